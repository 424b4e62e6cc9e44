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

constexpr int kWave = 1024;             // logits of a chunk: 16 of each lane
constexpr int kMaxNodes = 1024;

// Element k of a lane's 16 is number 256 (k / 4) + 4 lane + k % 4 of the chunk
__device__ __forceinline__ int chunk_index(int lane, int k) { return 256 * (k >> 2) + 4 * lane + (k & 3); }

// Four consecutive logits at p, of which `left` exist (NaN and what is missing: -inf)
template <typename T>
__device__ __forceinline__ void load4(const T *p, int64_t left, float v[4]) {
    if (left >= 4) {
        if constexpr (sizeof(T) == 2) {
            uint32_t w[2];
            __builtin_memcpy(w, p, 8);
            v[0] = __uint_as_float(w[0] << 16);
            v[1] = __uint_as_float(w[0] & 0xFFFF0000u);
            v[2] = __uint_as_float(w[1] << 16);
            v[3] = __uint_as_float(w[1] & 0xFFFF0000u);
        } else {
            __builtin_memcpy(v, p, 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < left ? load1<T>(p + i) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = v[i] == v[i] ? v[i] : -INFINITY;
}

template <typename T>
__device__ __forceinline__ void load_chunk(const T *row, int64_t V, int64_t at, int lane, float v[16]) {
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
        const int64_t i = at + chunk_index(lane, k);
        load4<T>(row + i, V - i, v + k);
    }
}

// exp((l - m) / T); l <= m. m = +inf leaves 1 where l is +inf too, m = -inf
// nothing; l = -inf is 0 at any T (at T = inf all other weights are 1)
__device__ __forceinline__ double weight(float l, float m, double inv) {
    const double e = exp(((double)l - (double)m) * inv);
    return l == -INFINITY ? 0.0 : (l == m ? 1.0 : (m == INFINITY ? 0.0 : e));
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ double wave_scan(double v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(v, o);
        if ((int)(threadIdx.x & 63) >= o) v += y;
    }
    return v;
}

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
    int C, max_n, replacement;
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

// A wave a chunk of a row: its maximum, and the sum of the weights against it
template <typename T>
__global__ __launch_bounds__(256) void k_row_stats(Args a) {
    const int lane = threadIdx.x & 63;
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * 65535;
    const int c = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= a.total || c >= a.C) return;
    double inv = 1.0;
    bool greedy = false;
    if (a.temperature) {
        const int64_t b = sequence_of(a, row, lane);
        if (b >= a.B) return;
        const float t = a.temperature[b];
        greedy = !(t > 0.f);
        inv = greedy ? 1.0 : 1.0 / (double)t;
    }
    float v[16];
    load_chunk<T>(static_cast<const T *>(a.logits) + row * a.ldl, a.V, (int64_t)c * kWave, lane, v);
    float m = v[0];
#pragma unroll
    for (int k = 1; k < 16; ++k) m = fmaxf(m, v[k]);
    m = wave_max(m);
    double s = 0.0;
    if (greedy) {
        int at = kWave;
#pragma unroll
        for (int k = 15; k >= 0; --k)
            if (v[k] == m) at = chunk_index(lane, k);
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            const int y = __shfl_xor(at, o);
            at = y < at ? y : at;
        }
        s = (double)((int64_t)c * kWave + at);
    } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) s += weight(v[k], m, inv);
        s = wave_sum(s);
    }
    if (lane == 0) {
        a.mx[row * a.C + c] = m;
        a.sum[row * a.C + c] = s;
    }
}

struct Walk {
    double S, R, left;
    int cur, i, kept, gone;             // node, next child to try, kept nodes, children of cur taken out (no draft)
    int done;
};

// One workgroup a sequence walks its tree. The walk itself is one thread's; the
// workgroup prepares what it reads (maximum and sum of every node's row, weight
// and draft probability of every token) and forms the sums of remainders.
template <typename T>
__global__ __launch_bounds__(1024) void k_walk(Args a) {
    __shared__ float node_m[kMaxNodes], node_q[kMaxNodes];
    __shared__ double node_z[kMaxNodes], node_e[kMaxNodes], node_u[kMaxNodes];
    __shared__ int node_p[kMaxNodes];
    __shared__ int node_best[kMaxNodes];
    __shared__ uint8_t node_out[kMaxNodes];       // taken out of its parent's row
    __shared__ Walk w;
    __shared__ double part[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t b = blockIdx.x;
    int c0 = a.cu[b], c1 = a.cu[b + 1];
    c0 = c0 < 0 ? 0 : c0;
    c1 = c1 > a.total ? (int)a.total : c1;
    const int rows = c1 > c0 ? c1 - c0 : 0;
    const int n = rows < a.max_n ? rows : a.max_n;
    if (n == 0) {
        for (int i = tid; i < rows; i += 1024) a.path[c0 + i] = -1;
        if (tid == 0) {
            a.count[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    const float t = a.temperature ? a.temperature[b] : 1.f;
    const bool greedy = !(t > 0.f);
    const double inv = greedy ? 1.0 : 1.0 / (double)t;
    const T *logits = static_cast<const T *>(a.logits) + (int64_t)c0 * a.ldl;
    const float *draft = a.draft && !greedy ? a.draft + (int64_t)c0 * a.ldd : nullptr;

    // maximum and sum of every row, from its chunks
    for (int i = wave; i < n; i += 16) {
        const float *mc = a.mx + (int64_t)(c0 + i) * a.C;
        const double *sc = a.sum + (int64_t)(c0 + i) * a.C;
        float m = -INFINITY;
        for (int c = lane; c < a.C; c += 64) m = fmaxf(m, mc[c]);
        m = wave_max(m);
        double z = 0.0;
        int best = 0x7FFFFFFF;
        for (int c = lane; c < a.C; c += 64) {
            if (greedy) {
                if (mc[c] == m && (int)sc[c] < best) best = (int)sc[c];
            } else {
                z += sc[c] * weight(mc[c], m, inv);
            }
        }
        z = wave_sum(z);
        for (int o = 32; o; o >>= 1) {
            const int y = __shfl_xor(best, o);
            best = y < best ? y : best;
        }
        if (lane == 0) {
            node_m[i] = m;
            node_z[i] = greedy ? (m == -INFINITY ? 0.0 : 1.0) : z;
            node_best[i] = m == -INFINITY ? -1 : best;
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += 1024) {
        const int p = a.parents ? a.parents[c0 + i] : i - 1;
        const int64_t x = a.tokens[c0 + i];
        const bool ok = i > 0 && p >= 0 && p < i && x >= 0 && x < a.V;
        double e = -1.0;                            // never accepted
        float q = 1.f;
        if (ok) {
            if (greedy) {
                e = x == node_best[p] ? 1.0 : 0.0;
            } else {
                float l = load1<T>(logits + p * a.ldl + x);
                l = l == l ? l : -INFINITY;
                e = weight(l, node_m[p], inv);
            }
            if (draft) {
                q = draft[p * a.ldd + x];
                q = q > 0.f && q < INFINITY ? q : 0.f;
            }
        }
        node_p[i] = i > 0 && p >= 0 && p < i ? p : -1;
        node_e[i] = e;
        node_q[i] = q;
        node_u[i] = a.uniform[c0 + i];
        node_out[i] = 0;
    }
    for (int i = tid; i < rows; i += 1024) a.path[c0 + i] = i == 0 ? 0 : -1;
    if (tid == 0) {
        w.S = 0.0;
        w.left = 1.0;
        w.cur = 0;
        w.i = 1;
        w.kept = 1;
        w.gone = 0;
        w.done = 0;
    }
    __syncthreads();
    if (tid == 0) w.R = node_z[0];
    double *rest = a.rest + b * a.C;
    for (;;) {
        if (tid == 0) {
            // until a remainder has to be summed, or no child is left
            int i = w.i, cur = w.cur;
            bool sum = false;
            for (; i < n && !sum; ++i) {
                if (node_p[i] != cur || node_e[i] < 0.0) continue;
                const double e = node_e[i], q = (double)node_q[i];
                bool ok;
                if (greedy) {
                    ok = e > 0.0;
                } else if (draft) {
                    const double r = e - w.S * q;
                    ok = w.left > 0.0 && node_u[i] * q * w.R < (r > 0.0 ? r : 0.0) * w.left;
                } else {
                    double r = e;
                    for (int j = cur + 1; j < i; ++j)             // the same token among its elder siblings
                        if (node_out[j] && node_p[j] == cur && a.tokens[c0 + j] == a.tokens[c0 + i]) r = 0.0;
                    ok = node_u[i] * w.R < r;
                    if (!ok && r > 0.0) {
                        node_out[i] = 1;
                        w.gone = 1;
                        w.R = w.R > r ? w.R - r : 0.0;
                    }
                }
                if (ok) {
                    a.path[c0 + w.kept] = i;
                    ++w.kept;
                    cur = i;
                    w.S = 0.0;
                    w.left = 1.0;
                    w.R = node_z[i];
                    w.gone = 0;
                } else if (draft && w.left > 0.0) {
                    w.S += w.R / w.left;
                    if (!a.replacement) w.left -= q;
                    sum = true;
                }
            }
            w.i = i;
            w.cur = cur;
            w.done = !sum;
        }
        __syncthreads();
        if (w.done) break;
        // the remainder's sum, chunk by chunk
        const T *row = logits + (int64_t)w.cur * a.ldl;
        const float *qrow = draft + (int64_t)w.cur * a.ldd;
        const float m = node_m[w.cur];
        const double S = w.S;
        for (int c = wave; c < a.C; c += 16) {
            float v[16], q[16];
            load_chunk<T>(row, a.V, (int64_t)c * kWave, lane, v);
            load_chunk<float>(qrow, a.V, (int64_t)c * kWave, lane, q);
            double s = 0.0;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const double qk = q[k] > 0.f && q[k] < INFINITY ? (double)q[k] : 0.0;
                const double r = weight(v[k], m, inv) - S * qk;
                s += r > 0.0 ? r : 0.0;
            }
            s = wave_sum(s);
            if (lane == 0) rest[c] = s;
        }
        __syncthreads();
        if (wave == 0) {
            double s = 0.0;
            for (int c = lane; c < a.C; c += 64) s += rest[c];
            s = wave_sum(s);
            if (lane == 0) w.R = s;
        }
        __syncthreads();
    }
    const int cur = w.cur;
    const float m = node_m[cur];
    if (tid == 0) a.count[b] = w.kept;
    if (greedy || node_z[cur] == 0.0) {
        if (tid == 0) a.next[b] = greedy ? node_best[cur] : -1;
        return;
    }
    // sums of the chunks of what is left: the target's own, less the tokens taken
    // out, unless a remainder was summed
    const bool rem = draft && w.S > 0.0;
    if (!rem) {
        for (int c = tid; c < a.C; c += 1024)
            rest[c] = a.sum[(int64_t)(c0 + cur) * a.C + c] * weight(a.mx[(int64_t)(c0 + cur) * a.C + c], m, inv);
        __syncthreads();
        if (tid == 0 && w.gone)
            for (int j = cur + 1; j < n; ++j)
                if (node_out[j] && node_p[j] == cur) {
                    const int c = (int)(a.tokens[c0 + j] / kWave);
                    const double r = rest[c] - node_e[j];
                    rest[c] = r > 0.0 ? r : 0.0;
                }
        __syncthreads();
    }
    if (wave != 0) return;
    // the first wave: total, chunk, token
    const int per = (a.C + 63) / 64;
    bool whole = false;                           // nothing left: the target's own weights
    for (;;) {
        double mine = 0.0;
        for (int c = lane * per; c < (lane + 1) * per && c < a.C; ++c)
            mine += whole ? a.sum[(int64_t)(c0 + cur) * a.C + c] * weight(a.mx[(int64_t)(c0 + cur) * a.C + c], m, inv) : rest[c];
        const double upto = wave_scan(mine);
        const double total = __shfl(upto, 63);
        if (!(total > 0.0) && !whole) {
            whole = true;
            continue;
        }
        const double target = node_u[0] * total;
        // first chunk whose inclusive sum is past the target, else the last one that holds anything
        int at = a.C, last = -1;
        double before = 0.0, run = upto - mine;
        for (int c = lane * per; c < (lane + 1) * per && c < a.C; ++c) {
            const double s = whole ? a.sum[(int64_t)(c0 + cur) * a.C + c] * weight(a.mx[(int64_t)(c0 + cur) * a.C + c], m, inv) : rest[c];
            if (s > 0.0) last = c;
            if (s > 0.0 && run + s > target && at == a.C) {
                at = c;
                before = run;
            }
            run += s;
        }
        const uint64_t found = __ballot(at < a.C);
        bool past = false;
        if (found) {
            const int f = __ffsll((long long)found) - 1;
            at = __shfl(at, f);
            before = __shfl(before, f);
        } else {
            const uint64_t any = __ballot(last >= 0);
            if (!any) {
                if (lane == 0) a.next[b] = -1;
                return;
            }
            at = __shfl(last, 63 - __clzll((long long)any));
            past = true;
        }
        // the token within the chunk
        float v[16], q[16];
        load_chunk<T>(logits + (int64_t)cur * a.ldl, a.V, (int64_t)at * kWave, lane, v);
        if (rem && !whole) load_chunk<float>(draft + (int64_t)cur * a.ldd, a.V, (int64_t)at * kWave, lane, q);
        double r[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int64_t x = (int64_t)at * kWave + chunk_index(lane, k);
            r[k] = weight(v[k], m, inv);
            if (rem && !whole) {
                const double qk = q[k] > 0.f && q[k] < INFINITY ? (double)q[k] : 0.0;
                r[k] -= w.S * qk;
                r[k] = r[k] > 0.0 ? r[k] : 0.0;
            }
            if (w.gone && !whole)
                for (int j = cur + 1; j < n; ++j)
                    if (node_out[j] && node_p[j] == cur && a.tokens[c0 + j] == x) r[k] = 0.0;
        }
        int64_t first = INT64_MAX, final_ = -1;
        double base = before;
#pragma unroll
        for (int g = 0; g < 4; ++g) {             // elements in the order of their index
            const double quad = ((r[4 * g] + r[4 * g + 1]) + r[4 * g + 2]) + r[4 * g + 3];
            const double inc = wave_scan(quad);
            double s = base + (inc - quad);
#pragma unroll
            for (int k = 4 * g; k < 4 * g + 4; ++k) {
                const int64_t x = (int64_t)at * kWave + chunk_index(lane, k);
                s += r[k];
                if (r[k] > 0.0) {
                    if (s > target && x < first) first = x;
                    if (x > final_) final_ = x;
                }
            }
            base += __shfl(inc, 63);
        }
        for (int o = 32; o; o >>= 1) {
            const int64_t y = __shfl_xor(first, o), z = __shfl_xor(final_, o);
            first = y < first ? y : first;
            final_ = z > final_ ? z : final_;
        }
        const int64_t x = past || first == INT64_MAX ? final_ : first;
        if (x < 0 && !whole) {                    // the chunk's sum was rounding alone
            whole = true;
            continue;
        }
        if (lane == 0) a.next[b] = x;
        return;
    }
}

size_t layout(int64_t B, int64_t total, int64_t V, size_t *sum, size_t *rest, int *C) {
    const int64_t c = ceil_div(V, (int64_t)kWave);
    const size_t mx = ((size_t)total * c * 4 + 15) / 16 * 16, s = (size_t)total * c * 8;
    if (sum) *sum = mx;
    if (rest) *rest = mx + s;
    if (C) *C = (int)c;
    return mx + s + (size_t)B * c * 8;
}

}  // namespace

size_t verify_tree_workspace(int64_t B, int64_t total, int64_t V) { return layout(B, total, V, nullptr, nullptr, nullptr); }

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
    size_t sum, rest;
    layout(B, total, V, &sum, &rest, &a.C);
    uint8_t *w = static_cast<uint8_t *>(ws);
    a.mx = reinterpret_cast<float *>(w);
    a.sum = reinterpret_cast<double *>(w + sum);
    a.rest = reinterpret_cast<double *>(w + rest);
    if (total > 0 && max_n > 0) {
        const dim3 grid((unsigned)ceil_div(a.C, 4), (unsigned)(total < 65535 ? total : 65535),
                        (unsigned)ceil_div(total, (int64_t)65535));
        if (dt == MXS_BF16) hipLaunchKernelGGL(k_row_stats<uint16_t>, grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL(k_row_stats<float>, grid, dim3(256), 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dt == MXS_BF16) hipLaunchKernelGGL(k_walk<uint16_t>, dim3((unsigned)B), dim3(1024), 0, st, a);
    else hipLaunchKernelGGL(k_walk<float>, dim3((unsigned)B), dim3(1024), 0, st, a);
    return hipGetLastError();
}

}  // namespace mxs
