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

constexpr int kChunkPages = 4096;       // pages of a bitmap chunk: 64 words of 64 bits

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

// ---------------------------------------------------------------------- copy
__global__ __launch_bounds__(256) void k_kv4_copy(Planes to, const int64_t *to_slots, Planes from,
                                                  const int64_t *from_slots, int64_t T) {
    const int nb = to.nb;
    const int64_t total = T * nb, step = (int64_t)gridDim.x * 256;
    const int p = blockIdx.y;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += step) {
        const int64_t t = e / nb;
        const int u = (int)(e - t * nb);
        const int64_t d = to_slots[t], s = from_slots[t];
        if ((uint64_t)d >= (uint64_t)to.slots || (uint64_t)s >= (uint64_t)from.slots) continue;
        reinterpret_cast<u32x4 *>(to.c[p])[d * nb + u] = reinterpret_cast<const u32x4 *>(from.c[p])[s * nb + u];
        to.s[p][d * nb + u] = from.s[p][s * nb + u];
    }
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
// Workspace: a bitmap of the free pages, their number in each chunk, the pages
// that each sequence needs (-1: its row is too short), and the pages granted.
struct Reserve {
    uint64_t *map;
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
    const size_t map = take(chunks * 64 * 8), counts = take(chunks * 4), need = take(B * 4), grant = take(pages * 4);
    if (r) {
        uint8_t *w = static_cast<uint8_t *>(ws);
        r->map = reinterpret_cast<uint64_t *>(w + map);
        r->counts = reinterpret_cast<int32_t *>(w + counts);
        r->need = reinterpret_cast<int32_t *>(w + need);
        r->grant = reinterpret_cast<int32_t *>(w + grant);
        r->chunks = (int)chunks;
    }
    return at;
}

__device__ __forceinline__ int wave_sum(int v) {
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
    if (len < 0 || (int64_t)len + n > a.ldt * a.page_size) return false;
    if (n == 0) return true;
    j0 = len / a.page_size;
    nj = ((int64_t)len + n - 1) / a.page_size - j0 + 1;
    return true;
}

// Waves of the first workgroups count what a sequence needs and mark entries
// whose page is shared by -2 - page (this decision stands while the second
// kernel changes refs); the others build the bitmap, a wave a chunk.
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
        int32_t *row = a.table + b * a.ldt;
        for (int64_t j = lane; j < nj; j += 64) {
            const int32_t p = row[j0 + j];
            const bool held = p >= 0 && p < a.pages;
            const bool shared = held && a.refs[p] > 1;
            if (shared) row[j0 + j] = -2 - p;
            else if (!held) row[j0 + j] = -1;
            need += !held || shared;
        }
        need = wave_sum(need);
        if (lane == 0) r.need[b] = need;
        return;
    }
    const int chunk = ((int)blockIdx.x - seq_groups) * 4 + wave;
    if (chunk >= r.chunks) return;
    uint64_t mine = 0;
    const int64_t p0 = (int64_t)chunk * kChunkPages;
    for (int k = 0; k < 64; ++k) {
        const int64_t p = p0 + k * 64 + lane;
        const uint64_t bits = __ballot(p < a.pages && a.refs[p < a.pages ? p : 0] == 0);
        if (lane == k) mine = bits;
    }
    r.map[(int64_t)chunk * 64 + lane] = mine;
    const int c = wave_sum(__popcll(mine));
    if (lane == 0) r.counts[chunk] = c;
}

// A workgroup a sequence: its ranks among the free pages, the pages themselves,
// then its table entries, the copy of a shared page's tokens, and its slots.
__global__ __launch_bounds__(256) void k_kv4_take(SeqArgs a, Reserve r, Planes pl, int64_t *slots, int32_t *lens_out) {
    __shared__ int part[256], sums[4], found[2], old_last, new_last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t b = blockIdx.x;
    int len, n;
    int64_t j0, nj;
    write_range(a, b, len, n, j0, nj);
    const int c0 = a.cu[b] < 0 ? 0 : a.cu[b];
    const int need = r.need[b];
    int32_t *row = a.table + b * a.ldt;
    // pages that earlier sequences need, and all that are free
    int before = 0, avail = 0;
    if (need > 0) {
        for (int64_t i = tid; i < b; i += 256) before += r.need[i] > 0 ? r.need[i] : 0;
        for (int i = tid; i < r.chunks; i += 256) avail += r.counts[i];
    }
    before = wave_sum(before);
    avail = wave_sum(avail);
    if (lane == 0) {
        sums[wave] = before;
        part[wave] = avail;
    }
    if (tid == 0) old_last = new_last = -1;
    __syncthreads();
    before = sums[0] + sums[1] + sums[2] + sums[3];
    avail = part[0] + part[1] + part[2] + part[3];
    __syncthreads();
    if (need < 0 || (need > 0 && (int64_t)before + need > avail)) {
        for (int64_t j = tid; j < nj; j += 256)
            if (row[j0 + j] < -1) row[j0 + j] = -2 - row[j0 + j];
        for (int i = tid; i < n; i += 256) slots[c0 + i] = -1;
        if (tid == 0) lens_out[b] = len;
        return;
    }
    if (need > 0) {
        // the chunk that holds rank `before`: each thread sums a run of chunks
        const int per = (r.chunks + 255) / 256;
        int s = 0;
        for (int i = tid * per; i < (tid + 1) * per && i < r.chunks; ++i) s += r.counts[i];
        part[tid] = s;
        __syncthreads();
        int up = 0;
        for (int i = 0; i < tid; ++i) up += part[i];
        if (up <= before && before < up + s) {
            int c = tid * per;
            while (up + r.counts[c] <= before) up += r.counts[c++];
            found[0] = c;
            found[1] = up;
        }
        __syncthreads();
        if (wave == 0) {
            int at = found[1];
            for (int c = found[0]; c < r.chunks && at < before + need; ++c) {
                uint64_t bits = r.map[(int64_t)c * 64 + lane];
                const int cnt = __popcll(bits), inc = wave_scan(cnt);
                int rank = at + inc - cnt;
                const int32_t p = c * kChunkPages + lane * 64;
                while (bits) {
                    const int k = __ffsll((long long)bits) - 1;
                    bits &= bits - 1;
                    if (rank >= before && rank < before + need) r.grant[rank] = p + k;
                    ++rank;
                }
                at += __shfl(inc, 63);
            }
        }
        __syncthreads();
        // entries in order take the granted pages in order
        int at = before;
        for (int64_t t0 = 0; t0 < nj; t0 += 256) {
            const int64_t j = t0 + tid;
            const int32_t v = j < nj ? row[j0 + j] : 0;
            const uint64_t takes = __ballot(v < 0);
            if (lane == 0) sums[wave] = __popcll(takes);
            __syncthreads();
            int rank = at + __popcll(takes & ((1ull << lane) - 1));
            for (int w = 0; w < wave; ++w) rank += sums[w];
            at += sums[0] + sums[1] + sums[2] + sums[3];
            if (v < 0) {
                const int32_t p = r.grant[rank];
                row[j0 + j] = p;
                a.refs[p] = 1;
                if (v < -1) {
                    atomicSub(a.refs + (-2 - v), 1);
                    if (j == 0) {
                        old_last = -2 - v;
                        new_last = p;
                    }
                }
            }
            __syncthreads();
        }
    }
    // tokens of the last page, before the new ones
    if (new_last >= 0) {
        const int64_t units = (int64_t)(len % a.page_size) * pl.nb;
        const int64_t from = (int64_t)old_last * a.page_size * pl.nb, to = (int64_t)new_last * a.page_size * pl.nb;
        for (int p = 0; p < 2; ++p)
            for (int64_t u = tid; u < units; u += 256) {
                reinterpret_cast<u32x4 *>(pl.c[p])[to + u] = reinterpret_cast<const u32x4 *>(pl.c[p])[from + u];
                pl.s[p][to + u] = pl.s[p][from + u];
            }
    }
    for (int i = tid; i < n; i += 256) {
        const int64_t t = (int64_t)len + i, j = t / a.page_size;
        slots[c0 + i] = (int64_t)row[j] * a.page_size + (t - j * a.page_size);
    }
    if (tid == 0) lens_out[b] = len + n;
}

// ------------------------------------------------------------------- compact
// A workgroup a sequence. Kept tokens are moved in ascending order, a thread a
// block column: number i lands where no later token is read, because path[i] >= i.
__global__ __launch_bounds__(256) void k_kv4_compact(SeqArgs a, Planes pl, const int32_t *path, const int32_t *count,
                                                     int32_t *lens_out) {
    const int64_t b = blockIdx.x;
    int len = a.lens[b], c0 = a.cu[b], c1 = a.cu[b + 1];
    c0 = c0 < 0 ? 0 : c0;
    c1 = c1 > a.total ? (int)a.total : c1;
    const int n = c1 > c0 ? c1 - c0 : 0;
    int kept = count[b];
    kept = kept < 0 ? 0 : (kept > n ? n : kept);
    const bool moves = len >= n;
    __syncthreads();                            // every thread has read lens before it may be written
    if (moves) {
        const int64_t base = (int64_t)len - n;
        const int32_t *row = a.table + b * a.ldt;
        auto slot = [&](int64_t t) -> int64_t {
            const int64_t j = t / a.page_size;
            const int32_t p = j < a.ldt ? row[j] : -1;
            return p < 0 || p >= a.pages ? -1 : (int64_t)p * a.page_size + (t - j * a.page_size);
        };
        for (int u = threadIdx.x; u < 2 * pl.nb; u += 256) {
            const int p = u >= pl.nb, w = p ? u - pl.nb : u;
            for (int i = 0; i < kept; ++i) {
                const int f = path[c0 + i];
                if (f <= i || f >= n) continue;
                const int64_t s = slot(base + f), d = slot(base + i);
                if (s < 0 || d < 0) continue;
                reinterpret_cast<u32x4 *>(pl.c[p])[d * pl.nb + w] = reinterpret_cast<const u32x4 *>(pl.c[p])[s * pl.nb + w];
                pl.s[p][d * pl.nb + w] = pl.s[p][s * pl.nb + w];
            }
        }
    }
    if (threadIdx.x == 0) lens_out[b] = moves ? len - n + kept : len;
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
    const int64_t g = ceil_div(T * to.nb, (int64_t)256);
    hipLaunchKernelGGL(k_kv4_copy, dim3((unsigned)(g < 65536 ? g : 65536), 2), dim3(256), 0, st, to, dst_slots, from,
                       src_slots, T);
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
                              int64_t total, int32_t *lens_out, hipStream_t st) {
    const SeqArgs a{nullptr, const_cast<int32_t *>(table), ldt, B, c.pages, total, lens, cu, c.page_size};
    hipLaunchKernelGGL(k_kv4_compact, dim3((unsigned)B), dim3(256), 0, st, a, planes_of(c), path, count, lens_out);
    return hipGetLastError();
}

hipError_t launch_kv4_release(const mxs_kv4_cache &c, int32_t *refs, int32_t *table, int64_t ldt, int64_t B,
                              const int32_t *lens, const int32_t *keep, int32_t *lens_out, hipStream_t st) {
    const SeqArgs a{refs, table, ldt, B, c.pages, 0, lens, nullptr, c.page_size};
    hipLaunchKernelGGL(k_kv4_release, dim3(row_groups(ldt), (unsigned)B), dim3(256), 0, st, a, keep, lens_out);
    return hipGetLastError();
}

}  // namespace mxs
