// mxs_pages.hip -- pages of the 4-bit K/V cache: tokens copied, sequences
// forked, room reserved, accepted tokens moved together, pages given back.
//
// A block of 32 values is 16 bytes of codes and one scale byte, so a token of
// H heads of D values has nb = H D / 32 code words of 16 bytes and nb scale
// bytes in each of the planes K and V. Bytes are moved as they are. Pages are
// counted by integer atomics, whose order does not matter; which page an entry
// takes depends on ranks alone.
#include "mxs_device.h"
#include "mxs_internal.h"

namespace mxs {

namespace {

constexpr int kChunkPages = 1024;       // pages of a bitmap chunk: 16 of each lane

struct Planes {
    uint8_t *c[2], *s[2];               // codes and scales of K and V
    int64_t slots;
    int nb;                             // 32-blocks of a token and plane
};

Planes planes_of(const mxs_kv4_cache &c) {
    Planes p;
    p.c[0] = c.kc; p.c[1] = c.vc;
    p.s[0] = c.ks; p.s[1] = c.vs;
    p.slots = c.pages * c.page_size;
    p.nb = c.H * (c.D / 32);
    return p;
}

// n / d for n < 65536, d <= 65536: m = ceil(2^32 / d), 0 for d = 1
struct Div16 {
    uint32_t m, d;
};
Div16 div16(uint32_t d) { return Div16{d <= 1 ? 0u : (uint32_t)((0x100000000ull + d - 1) / d), d ? d : 1u}; }
__device__ __forceinline__ uint32_t quot(uint32_t n, Div16 v) { return v.m ? __umulhi(n, v.m) : n; }

// ---------------------------------------------------------------------- copy
// Bound by HBM: 131072 tokens of 8 heads of 128 take 59 us (4.9 TB/s, the rate of
// a plain copy). A workgroup takes whole tokens of one plane, or a chunk of one: WPT
// code words a thread, loaded before the first is stored, and their scale bytes,
// eight at a time where a token has a multiple of eight. Four words a thread pass the
// caches by (68 us if not); one, where the tokens are few, does not.
template <bool WIDE, int WPT>
__global__ __launch_bounds__(256) void k_kv4_copy(Planes to, const int64_t *to_slots, Planes from,
                                                  const int64_t *from_slots, int64_t T, int TB, Div16 chunk) {
    const int nb = to.nb, p = blockIdx.y;
    const int64_t t0 = (int64_t)blockIdx.x * TB;
    const int nt = T - t0 < TB ? (int)(T - t0) : TB;
    const uint32_t w0 = blockIdx.z * chunk.d;
    int64_t d[WPT], s[WPT];
    u32x4 v[WPT];
    uint8_t b[WPT];
#pragma unroll
    for (int k = 0; k < WPT; ++k) {
        const uint32_t e = threadIdx.x + 256u * k, tl = quot(e, chunk), w = w0 + e - tl * chunk.d;
        const bool on = tl < (uint32_t)nt && w < (uint32_t)nb;
        d[k] = on ? to_slots[t0 + tl] : -1;
        s[k] = on ? from_slots[t0 + tl] : -1;
        if ((uint64_t)d[k] >= (uint64_t)to.slots || (uint64_t)s[k] >= (uint64_t)from.slots) d[k] = -1;
        d[k] = d[k] < 0 ? -1 : d[k] * nb + w;
        s[k] = s[k] * nb + w;
    }
#pragma unroll
    for (int k = 0; k < WPT; ++k)
        if (d[k] >= 0) {
            const u32x4 *x = reinterpret_cast<const u32x4 *>(from.c[p]) + s[k];
            v[k] = WPT > 1 ? __builtin_nontemporal_load(x) : *x;
            if constexpr (!WIDE) b[k] = from.s[p][s[k]];
        }
    uint64_t wide = 0;
    int64_t wd = -1;
    if constexpr (WIDE) {
        const uint32_t e = 8u * threadIdx.x, tl = quot(e, chunk), w = w0 + e - tl * chunk.d;
        if (e < 256 * WPT && tl < (uint32_t)nt && w < (uint32_t)nb) {
            const int64_t td = to_slots[t0 + tl], ts = from_slots[t0 + tl];
            if ((uint64_t)td < (uint64_t)to.slots && (uint64_t)ts < (uint64_t)from.slots) {
                wd = td * nb + w;
                wide = *reinterpret_cast<const uint64_t *>(from.s[p] + ts * nb + w);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < WPT; ++k)
        if (d[k] >= 0) {
            u32x4 *x = reinterpret_cast<u32x4 *>(to.c[p]) + d[k];
            if constexpr (WPT > 1) __builtin_nontemporal_store(v[k], x);
            else *x = v[k];
            if constexpr (!WIDE) to.s[p][d[k]] = b[k];
        }
    if (WIDE && wd >= 0) *reinterpret_cast<uint64_t *>(to.s[p] + wd) = wide;
}

template <int WPT>
void copy_go(const Planes &to, const int64_t *to_slots, const Planes &from, const int64_t *from_slots, int64_t T,
             hipStream_t st) {
    const int nb = to.nb, most = 256 * WPT, tb = nb < most ? most / nb : 1;
    const Div16 chunk = div16(nb < most ? nb : most);
    const dim3 grid((unsigned)ceil_div(T, (int64_t)tb), 2, (unsigned)ceil_div(nb, (int64_t)chunk.d));
    if (nb % 8 == 0)
        hipLaunchKernelGGL((k_kv4_copy<true, WPT>), grid, dim3(256), 0, st, to, to_slots, from, from_slots, T, tb, chunk);
    else
        hipLaunchKernelGGL((k_kv4_copy<false, WPT>), grid, dim3(256), 0, st, to, to_slots, from, from_slots, T, tb, chunk);
}

// ---------------------------------------------------------------------- fork
__global__ __launch_bounds__(256) void k_kv4_fork(int32_t *refs, int32_t *table, int64_t ldt, int64_t B,
                                                  int32_t *lens, const int32_t *src, const int32_t *dst,
                                                  int64_t pages, int page_size) {
    const int s = src[blockIdx.y], d = dst[blockIdx.y];
    if (s < 0 || s >= B || d < 0 || d >= B || s == d) return;
    const int len = lens[s];
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < ldt; j += (int64_t)gridDim.x * 256) {
        int32_t p = j * page_size < len ? table[s * ldt + j] : -1;
        if (p < 0 || p >= pages) p = -1;
        else atomicAdd(refs + p, 1);
        table[d * ldt + j] = p;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) lens[d] = len;
}

// ------------------------------------------------------------------- reserve
// Workspace: bitmaps of the free and of the shared pages, the number of free ones in
// each chunk, the pages that each sequence needs (-1: its row is too short), and the
// pages granted.
struct Reserve {
    uint16_t *map, *shared;
    int32_t *counts, *need, *grant;
    int chunks;
};

size_t reserve_layout(int64_t pages, int64_t B, void *ws, Reserve *r) {
    const int64_t chunks = ceil_div(pages, (int64_t)kChunkPages);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 15) / 16 * 16;
        return o;
    };
    const size_t map = take(chunks * 64 * 2), shared = take(chunks * 64 * 2), counts = take(chunks * 4), need = take(B * 4), grant = take(pages * 4);
    if (r) {
        uint8_t *w = static_cast<uint8_t *>(ws);
        r->map = reinterpret_cast<uint16_t *>(w + map);
        r->shared = reinterpret_cast<uint16_t *>(w + shared);
        r->counts = reinterpret_cast<int32_t *>(w + counts);
        r->need = reinterpret_cast<int32_t *>(w + need);
        r->grant = reinterpret_cast<int32_t *>(w + grant);
        r->chunks = (int)chunks;
    }
    return at;
}

template <typename I>
__device__ __forceinline__ I wave_sum(I v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
// inclusive sum over the lanes up to this one
__device__ __forceinline__ int wave_scan(int v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(v, o);
        if ((int)(threadIdx.x & 63) >= o) v += y;
    }
    return v;
}

struct SeqArgs {
    int32_t *refs, *table;
    int64_t ldt, B, pages, total;
    const int32_t *lens, *cu;
    int page_size;
};

// First table entry and number of entries that sequence b writes to; false if its row is too short
__device__ __forceinline__ bool write_range(const SeqArgs &a, int64_t b, int &len, int &n, int64_t &j0, int64_t &nj) {
    len = a.lens[b];
    int c0 = a.cu[b], c1 = a.cu[b + 1];
    c0 = c0 < 0 ? 0 : c0;
    c1 = c1 > a.total ? (int)a.total : c1;
    n = c1 > c0 ? c1 - c0 : 0;
    j0 = nj = 0;
    if (len < 0 || (int64_t)len + n > a.ldt * a.page_size || (int64_t)len + n > 0x7FFFFFFF) return false;
    if (n == 0) return true;
    j0 = len / a.page_size;
    nj = ((int64_t)len + n - 1) / a.page_size - j0 + 1;
    return true;
}

// Latency bounds both kernels of a reservation: 2.4 + 8.3 us for two sequences over 64
// pages, 3.3 + 9.3 for 96 over 16384, 64 of which copy half a page (70 KB). A prompt's
// slots are written by its workgroup alone, one a thread and turn: 9.3 us for eight of
// 4096 tokens, 119 for one of 131072.
// Waves of the first workgroups count what a sequence needs; the others build the
// bitmaps, a wave a chunk. Which pages were shared is read from there while the second
// kernel changes refs, so no entry is written before its page is granted.
__global__ __launch_bounds__(256) void k_kv4_need(SeqArgs a, Reserve r, int seq_groups) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if ((int)blockIdx.x < seq_groups) {
        const int64_t b = (int64_t)blockIdx.x * 4 + wave;
        if (b >= a.B) return;
        int len, n;
        int64_t j0, nj;
        if (!write_range(a, b, len, n, j0, nj)) {
            if (lane == 0) r.need[b] = -1;
            return;
        }
        int need = 0;
        const int32_t *row = a.table + b * a.ldt;
        for (int64_t j = lane; j < nj; j += 64) {
            const int32_t p = row[j0 + j];
            const bool held = p >= 0 && p < a.pages;
            need += !held || a.refs[p] > 1;
        }
        need = wave_sum(need);
        if (lane == 0) r.need[b] = need;
        return;
    }
    const int chunk = ((int)blockIdx.x - seq_groups) * 4 + wave;
    if (chunk >= r.chunks) return;
    // 16 pages a lane, all loaded at once
    const int64_t p0 = (int64_t)chunk * kChunkPages + 16 * lane;
    uint32_t mine = 0, many = 0;
    if (p0 + 16 <= a.pages) {
        int4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) __builtin_memcpy(&v[k], a.refs + p0 + 4 * k, 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mine |= ((v[k].x == 0) | (v[k].y == 0) << 1 | (v[k].z == 0) << 2 | (v[k].w == 0) << 3) << 4 * k;
            many |= ((v[k].x > 1) | (v[k].y > 1) << 1 | (v[k].z > 1) << 2 | (v[k].w > 1) << 3) << 4 * k;
        }
    } else {
#pragma unroll 1
        for (int k = 0; k < 16 && p0 + k < a.pages; ++k) {
            const int32_t v = a.refs[p0 + k];
            mine |= (uint32_t)(v == 0) << k;
            many |= (uint32_t)(v > 1) << k;
        }
    }
    r.map[(int64_t)chunk * 64 + lane] = (uint16_t)mine;
    r.shared[(int64_t)chunk * 64 + lane] = (uint16_t)many;
    const int c = wave_sum(__popc(mine));
    if (lane == 0) r.counts[chunk] = c;
}

// n bytes, a multiple of 16, at 16-byte places; the loads of a turn go before its stores
__device__ __forceinline__ void copy16(uint8_t *to, const uint8_t *from, int64_t n) {
    for (int64_t e = 16 * threadIdx.x; e < n; e += 16 * 1024) {
        u32x4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e + 4096 * k < n) v[k] = *reinterpret_cast<const u32x4 *>(from + e + 4096 * k);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (e + 4096 * k < n) *reinterpret_cast<u32x4 *>(to + e + 4096 * k) = v[k];
    }
}
// n bytes at any places
__device__ __forceinline__ void copy_bytes(uint8_t *to, const uint8_t *from, int64_t n) {
    int64_t done = 0;
    if ((reinterpret_cast<uintptr_t>(to) | reinterpret_cast<uintptr_t>(from)) % 8 == 0) {
        done = n / 8 * 8;
        for (int64_t e = 8 * threadIdx.x; e < done; e += 8 * 256)
            *reinterpret_cast<uint64_t *>(to + e) = *reinterpret_cast<const uint64_t *>(from + e);
    }
    for (int64_t e = done + threadIdx.x; e < n; e += 256) to[e] = from[e];
}

// A workgroup a sequence: its ranks among the free pages, the pages themselves,
// then its table entries, its slots, and the copy of a shared page's tokens.
__global__ __launch_bounds__(256) void k_kv4_take(SeqArgs a, Reserve r, Planes pl, int64_t *slots, int32_t *lens_out) {
    __shared__ int64_t needs[4];
    __shared__ int sums[2][4], found[2], old_last, new_last;
    __shared__ int32_t few[256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t b = blockIdx.x;
    int len, n;
    int64_t j0, nj;
    write_range(a, b, len, n, j0, nj);
    const int c0 = a.cu[b] < 0 ? 0 : a.cu[b];
    const int need = r.need[b];
    int32_t *row = a.table + b * a.ldt;
    if (tid == 0) old_last = new_last = -1;
    __syncthreads();                            // every thread has read lens before it may be written
    int64_t wanted = 0;                         // 64 bits: no lens and cu make it wrap
    int avail = 0, mine = 0, upto = 0;
    const int per = (r.chunks + 255) / 256;
    // entries of the first turn and whether they take a page, loaded before anything waits
    auto entry = [&](int64_t j, bool &takes) {
        const int32_t p = j < nj ? row[j0 + j] : 0;
        const bool held = p >= 0 && p < a.pages;
        takes = j < nj && (!held || (r.shared[p >> 4] >> (p & 15) & 1));
        return held ? p : -1;
    };
    bool takes = false;
    int32_t page = -1;
    if (need > 0) {
        page = entry(tid, takes);
        // pages that earlier sequences need, and all that are free, a run of chunks a thread
        for (int64_t i = tid; i < b; i += 256) wanted += r.need[i] > 0 ? r.need[i] : 0;
        for (int i = tid * per; i < (tid + 1) * per && i < r.chunks; ++i) mine += r.counts[i];
        wanted = wave_sum(wanted);
        upto = wave_scan(mine);
        if (lane == 63) {
            needs[wave] = wanted;
            sums[0][wave] = upto;
        }
        __syncthreads();
        wanted = needs[0] + needs[1] + needs[2] + needs[3];
        avail = sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3];
        for (int w = 0; w < wave; ++w) upto += sums[0][w];
    }
    if (need < 0 || (need > 0 && wanted + need > avail)) {
        for (int i = tid; i < n; i += 256) slots[c0 + i] = -1;
        if (tid == 0) lens_out[b] = len;
        return;
    }
    const int before = (int)wanted;             // at most the free pages
    if (need > 0) {
        // the chunk that holds rank `before`, then the pages of the ranks from there
        if (upto - mine <= before && before < upto) {
            int c = tid * per, up = upto - mine;
            while (up + r.counts[c] <= before) up += r.counts[c++];
            found[0] = c;
            found[1] = up;
        }
        __syncthreads();
        int32_t *grant = need <= 256 ? few : r.grant + before;
        if (wave == 0) {
            int at = found[1] - before;
            for (int c = found[0]; c < r.chunks && at < need; ++c) {
                uint32_t bits = r.map[(int64_t)c * 64 + lane];
                const int cnt = __popc(bits), inc = wave_scan(cnt);
                int rank = at + inc - cnt;
                const int32_t p = c * kChunkPages + lane * 16;
                while (bits) {
                    const int k = __ffs((int)bits) - 1;
                    bits &= bits - 1;
                    if (rank >= 0 && rank < need) grant[rank] = p + k;
                    ++rank;
                }
                at += __shfl(inc, 63);
            }
        }
        __syncthreads();
        // entries in order take the granted pages in order
        int at = 0;
        for (int64_t t0 = 0; t0 < nj; t0 += 256) {
            const int64_t j = t0 + tid;
            if (t0 > 0) page = entry(j, takes);
            const uint64_t who = __ballot(takes);
            if (lane == 0) sums[1][wave] = __popcll(who);
            __syncthreads();
            int rank = at + __popcll(who & ((1ull << lane) - 1));
            for (int w = 0; w < wave; ++w) rank += sums[1][w];
            at += sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3];
            if (takes) {
                const int32_t p = grant[rank];
                row[j0 + j] = p;
                a.refs[p] = 1;
                if (page >= 0) {
                    atomicSub(a.refs + page, 1);
                    if (j == 0) {
                        old_last = page;
                        new_last = p;
                    }
                }
            }
            __syncthreads();
        }
    }
    for (int i = tid; i < n; i += 256) {
        const int64_t t = (int64_t)len + i, j = t / a.page_size;
        slots[c0 + i] = (int64_t)row[j] * a.page_size + (t - j * a.page_size);
    }
    if (tid == 0) lens_out[b] = len + n;
    // tokens of a shared last page before the new ones: one run of bytes a plane
    if (need > 0 && new_last >= 0) {
        const int64_t units = (int64_t)(len % a.page_size) * pl.nb, unit = (int64_t)a.page_size * pl.nb;
        for (int p = 0; p < 2; ++p) {
            copy16(pl.c[p] + 16 * new_last * unit, pl.c[p] + 16 * old_last * unit, 16 * units);
            copy_bytes(pl.s[p] + new_last * unit, pl.s[p] + old_last * unit, units);
        }
    }
}

// ------------------------------------------------------------------- compact
// A workgroup a sequence. The slots of 256 kept tokens are found first, then tokens
// are moved 1024 code words (with their scale bytes) at a time, in ascending
// order: all are read before the first is written, and what a later turn reads no
// earlier one has written, because path[i] >= i. 96 sequences of up to 26 tokens take
// 6.0 us (a thread a column, token after token: 15). A sequence whose first slot is -1
// was refused its tokens: its last ones are not theirs, and may lie in shared pages.
__global__ __launch_bounds__(256) void k_kv4_compact(SeqArgs a, Planes pl, const int32_t *path, const int32_t *count,
                                                     const int64_t *slots, int32_t *lens_out) {
    __shared__ int32_t from[256], to[256];
    const int64_t b = blockIdx.x;
    const int tid = threadIdx.x;
    int len = a.lens[b], c0 = a.cu[b], c1 = a.cu[b + 1];
    c0 = c0 < 0 ? 0 : c0;
    c1 = c1 > a.total ? (int)a.total : c1;
    const int n = c1 > c0 ? c1 - c0 : 0;
    int kept = count[b];
    kept = kept < 0 ? 0 : (kept > n ? n : kept);
    const bool moves = len >= n && !(slots && n > 0 && slots[c0] < 0);
    __syncthreads();                            // every thread has read lens before it may be written
    if (tid == 0) lens_out[b] = moves ? len - n + kept : len;
    if (!moves) return;
    const int64_t base = (int64_t)len - n;
    const int32_t *row = a.table + b * a.ldt;
    auto slot = [&](int64_t t) -> int32_t {
        const int64_t j = t / a.page_size;
        const int32_t p = j < a.ldt ? row[j] : -1;
        return p < 0 || p >= a.pages ? -1 : (int32_t)(p * a.page_size + (t - j * a.page_size));
    };
    const int words = 2 * pl.nb;                // of a token: K's, then V's
    for (int i0 = 0; i0 < kept; i0 += 256) {
        const int m = kept - i0 < 256 ? kept - i0 : 256;
        if (tid < m) {
            const int f = path[c0 + i0 + tid];
            const bool on = f > i0 + tid && f < n;
            const int32_t s = on ? slot(base + f) : -1, d = on ? slot(base + i0 + tid) : -1;
            from[tid] = d < 0 ? -1 : s;
            to[tid] = d;
        }
        __syncthreads();
        for (int64_t e0 = 0; e0 < (int64_t)m * words; e0 += 1024) {
            u32x4 v[4];
            uint8_t sc[4];
            int64_t d[4];
            int pk[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t e = e0 + tid + 256 * k;
                d[k] = -1;
                if (e < (int64_t)m * words) {
                    const int i = (int)(e / words), u = (int)(e - (int64_t)i * words), p = u >= pl.nb, w = p ? u - pl.nb : u;
                    const int32_t s = from[i];
                    if (s >= 0) {
                        pk[k] = p;
                        d[k] = (int64_t)to[i] * pl.nb + w;
                        v[k] = reinterpret_cast<const u32x4 *>(pl.c[p])[(int64_t)s * pl.nb + w];
                        sc[k] = pl.s[p][(int64_t)s * pl.nb + w];
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (d[k] >= 0) {
                    reinterpret_cast<u32x4 *>(pl.c[pk[k]])[d[k]] = v[k];
                    pl.s[pk[k]][d[k]] = sc[k];
                }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------- release
__global__ __launch_bounds__(256) void k_kv4_release(SeqArgs a, const int32_t *keep, int32_t *lens_out) {
    const int64_t b = blockIdx.y;
    const int k = keep[b];
    if (k >= 0) {
        const int64_t j0 = ((int64_t)k + a.page_size - 1) / a.page_size;
        for (int64_t j = j0 + (int64_t)blockIdx.x * 256 + threadIdx.x; j < a.ldt; j += (int64_t)gridDim.x * 256) {
            const int32_t p = a.table[b * a.ldt + j];
            if (p >= 0 && p < a.pages) atomicSub(a.refs + p, 1);
            a.table[b * a.ldt + j] = -1;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        const int len = a.lens[b];
        lens_out[b] = k >= 0 && k < len ? k : len;
    }
}

unsigned row_groups(int64_t ldt) {
    const int64_t g = ceil_div(ldt, (int64_t)256);
    return (unsigned)(g < 1 ? 1 : (g > 64 ? 64 : g));
}

}  // namespace

size_t kv4_reserve_workspace(int64_t pages, int64_t B) { return reserve_layout(pages, B, nullptr, nullptr); }

hipError_t launch_kv4_copy(const mxs_kv4_cache &dst, const int64_t *dst_slots, const mxs_kv4_cache &src,
                           const int64_t *src_slots, int64_t T, hipStream_t st) {
    const Planes to = planes_of(dst), from = planes_of(src);
    // one word a thread until the chip is full four times over (as the append): 2.6
    // against 4.2 us at 1901 tokens of 3 heads of 96
    if (2 * T * to.nb < 4 * 256 * 2048) copy_go<1>(to, dst_slots, from, src_slots, T, st);
    else copy_go<4>(to, dst_slots, from, src_slots, T, st);
    return hipGetLastError();
}

hipError_t launch_kv4_fork(const mxs_kv4_cache &c, int32_t *refs, int32_t *table, int64_t ldt, int64_t B,
                           int32_t *lens, const int32_t *src, const int32_t *dst, int64_t n, hipStream_t st) {
    hipLaunchKernelGGL(k_kv4_fork, dim3(row_groups(ldt), (unsigned)n), dim3(256), 0, st, refs, table, ldt, B, lens,
                       src, dst, c.pages, c.page_size);
    return hipGetLastError();
}

hipError_t launch_kv4_reserve(const mxs_kv4_cache &c, int32_t *refs, int32_t *table, int64_t ldt, int64_t B,
                              const int32_t *lens, const int32_t *cu, int64_t total, int64_t *slots,
                              int32_t *lens_out, void *ws, hipStream_t st) {
    Reserve r;
    reserve_layout(c.pages, B, ws, &r);
    const SeqArgs a{refs, table, ldt, B, c.pages, total, lens, cu, c.page_size};
    const int groups = (int)ceil_div(B, (int64_t)4);
    hipLaunchKernelGGL(k_kv4_need, dim3(groups + (unsigned)ceil_div(r.chunks, 4)), dim3(256), 0, st, a, r, groups);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_kv4_take, dim3((unsigned)B), dim3(256), 0, st, a, r, planes_of(c), slots, lens_out);
    return hipGetLastError();
}

hipError_t launch_kv4_compact(const mxs_kv4_cache &c, const int32_t *table, int64_t ldt, int64_t B,
                              const int32_t *lens, const int32_t *cu, const int32_t *path, const int32_t *count,
                              const int64_t *slots, int64_t total, int32_t *lens_out, hipStream_t st) {
    const SeqArgs a{nullptr, const_cast<int32_t *>(table), ldt, B, c.pages, total, lens, cu, c.page_size};
    hipLaunchKernelGGL(k_kv4_compact, dim3((unsigned)B), dim3(256), 0, st, a, planes_of(c), path, count, slots, lens_out);
    return hipGetLastError();
}

hipError_t launch_kv4_release(const mxs_kv4_cache &c, int32_t *refs, int32_t *table, int64_t ldt, int64_t B,
                              const int32_t *lens, const int32_t *keep, int32_t *lens_out, hipStream_t st) {
    const SeqArgs a{refs, table, ldt, B, c.pages, 0, lens, nullptr, c.page_size};
    hipLaunchKernelGGL(k_kv4_release, dim3(row_groups(ldt), (unsigned)B), dim3(256), 0, st, a, keep, lens_out);
    return hipGetLastError();
}

}  // namespace mxs
