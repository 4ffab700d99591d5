// Attention of a few tokens per sequence against a paged cache, with prefixes that groups of sequences share
// (gdr_attn_decode_paged).
//
// The tokens of one sequence (or, over a shared prefix, of a whole group) times the query heads of one key head
// are the rows of one product: keys and values are read once for all of them.  The work is a line of tiles of 64
// keys, (key head, unit, row block, tile) in that order, cut into equal stretches for a fixed number of
// workgroups, whatever the lengths are: the host does not know them.  A stretch may end inside a unit; such a
// part's maximum, sum and unnormalised output go to the workspace and are joined by the last kernel.
//   attn_plan_kernel   the units' tiles summed up (one workgroup)
//   attn_paged_kernel  the groups' prefixes, then what is each sequence's own
//   attn_join_kernel   parts -> outputs
#include <hip/hip_runtime.h>

#include "gdr_attn_device.h"

namespace gdr {
namespace {

constexpr int kKeys = 64;       // keys per tile
constexpr int kMinTiles = 2;    // tiles of a workgroup's stretch at least: below, parts cost more than they save

__device__ __forceinline__ int seq_first(const AttnPagedArgs& a, int n) { return a.cu ? a.cu[n] : n; }

// keys that a sequence's last token sees; 0 for a padded sequence and one without tokens
__device__ __forceinline__ int seq_keys(const AttnPagedArgs& a, int n) {
    const int ctx = a.context[n], count = a.cu ? a.cu[n + 1] - a.cu[n] : 1;
    if (ctx < 0 || count <= 0) return 0;
    return (int)min((int64_t)ctx + count, a.capacity);
}

__device__ __forceinline__ int64_t stretch(const AttnPagedArgs& a, int64_t tiles) {
    return max((tiles + a.workers - 1) / a.workers, (int64_t)kMinTiles);
}

// Sums up the units' tiles and row blocks.  One workgroup; every thread takes a run of units.
__global__ __launch_bounds__(1024) void attn_plan_kernel(AttnPagedArgs a) {
    __shared__ int64_t tiles[1024];
    __shared__ int items[1024];
    const int tid = threadIdx.x;
    for (int n = tid; n < a.N; n += 1024) { a.pre[n] = 0; a.group[n] = -1; }
    __syncthreads();
    // groups: the first sequence that is not padded gives the pages, whole pages are shared
    for (int g = tid; g < a.groups; g += 1024) {
        const int s = max(0, min(a.group_offsets[g], a.N)), e = max(s, min(a.group_offsets[g + 1], a.N));
        int rep = -1;
        for (int n = s; n < e && rep < 0; ++n)
            if (seq_keys(a, n) > 0) rep = n;
        const int64_t len = rep < 0 ? 0 : min((int64_t)max(0, a.prefix_lens[g]), a.capacity);
        const int pre = (int)(len >> a.page_shift << a.page_shift);
        a.rep[g] = rep;
        a.prefix[g] = pre;
        for (int n = s; n < e; ++n) { a.pre[n] = pre; a.group[n] = g; }
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        const int units = side == 0 ? a.N : a.groups;
        const int rows = side == 0 ? a.rows : a.prefix_rows;
        int64_t* cum = side == 0 ? a.cum : a.prefix_cum;
        int* item = side == 0 ? a.item : a.prefix_item;
        auto unit = [&](int u, int64_t* t, int* i) {
            int keys, tokens;
            if (side == 0) {
                keys = max(0, seq_keys(a, u) - a.pre[u]);
                tokens = a.cu ? a.cu[u + 1] - a.cu[u] : 1;
            } else {
                const int s = max(0, min(a.group_offsets[u], a.N)), e = max(s, min(a.group_offsets[u + 1], a.N));
                keys = a.prefix[u];
                tokens = seq_first(a, e) - seq_first(a, s);
            }
            const int blocks = (int)(((int64_t)tokens * a.per + rows - 1) / rows);
            *i = keys > 0 ? blocks : 0;
            *t = (int64_t)*i * ((keys + kKeys - 1) / kKeys);
        };
        const int run = (units + 1023) / 1024, u0 = tid * run, u1 = min(u0 + run, units);
        int64_t st = 0;
        int si = 0;
        for (int u = u0; u < u1; ++u) {
            int64_t t; int i;
            unit(u, &t, &i);
            st += t; si += i;
        }
        tiles[tid] = st;
        items[tid] = si;
        __syncthreads();
        for (int d = 1; d < 1024; d *= 2) {
            const int64_t t = tid >= d ? tiles[tid - d] : 0;
            const int i = tid >= d ? items[tid - d] : 0;
            __syncthreads();
            tiles[tid] += t;
            items[tid] += i;
            __syncthreads();
        }
        st = tiles[tid] - st;
        si = items[tid] - si;
        for (int u = u0; u < u1; ++u) {
            int64_t t; int i;
            unit(u, &t, &i);
            cum[u] = st; item[u] = si;
            st += t; si += i;
        }
        if (tid == 1023) { cum[units] = tiles[1023]; item[units] = items[1023]; }
        __syncthreads();
    }
}

// last u with cum[u] <= y (so an empty unit is never found), 64 candidates at a time
__device__ __forceinline__ int find_unit(const int64_t* cum, int units, int64_t y) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = units;   // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int at = lo + lane * step;
        const bool yes = at < lo + n && cum[at] <= y;
        const int k = __popcll(__ballot(yes)) - 1;
        const int nlo = lo + k * step;
        n = min(step, lo + n - nlo);
        lo = nlo;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

struct Unit {
    int tok0, rows;      // first token, tokens * heads per key head
    int key0, key1;      // keys
    int table;           // row of the page table
    int tiles;
};

__device__ __forceinline__ Unit unit_of(const AttnPagedArgs& a, bool prefix, int u) {
    Unit r;
    if (prefix) {
        const int s = max(0, min(a.group_offsets[u], a.N)), e = max(s, min(a.group_offsets[u + 1], a.N));
        r.tok0 = seq_first(a, s);
        r.rows = (seq_first(a, e) - r.tok0) * a.per;
        r.key0 = 0;
        r.key1 = a.prefix[u];
        r.table = a.rep[u];
    } else {
        r.tok0 = seq_first(a, u);
        r.rows = (seq_first(a, u + 1) - r.tok0) * a.per;
        r.key0 = a.pre[u];
        r.key1 = seq_keys(a, u);
        r.table = u;
    }
    r.tiles = (r.key1 - r.key0 + kKeys - 1) / kKeys;
    return r;
}

// Parts of unit u's row block: the slots they are in.  A unit's block that one stretch holds whole is one part,
// in its own slot (or nowhere: it was written straight to the output).
__device__ __forceinline__ int64_t open_slot(int64_t w, bool continued) { return 2 * w + (continued ? 0 : 1); }

template <typename T, int D, int KW, int RW>
__global__ __launch_bounds__(64 * KW * RW) void attn_paged_kernel(AttnPagedArgs a, bool prefix) {
    using L = AttnTile<T, D>;
    using C = AttnCore<T, D>;
    constexpr int WAVES = KW * RW, blocks = 2 / KW;
    __shared__ __align__(1024) char lds[2 * kKeys * L::row_bytes];
    const uint32_t sk = lds_address(lds), sv = sk + kKeys * L::row_bytes;
    __shared__ float xch[KW == 2 ? RW * 64 * 18 : 1];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    const int kw = wave % KW, rw = wave / KW;
    const typename C::At at_(lds_address(lds), lds_address(lds) + kKeys * L::row_bytes, lane);
    const int64_t* cum = prefix ? a.prefix_cum : a.cum;
    const int* item = prefix ? a.prefix_item : a.item;
    const int units = prefix ? a.groups : a.N;
    char* const slots = prefix ? a.prefix_slots : a.slots;
    const int64_t slot_bytes = (int64_t)(32 * RW) * (D + 2) * 4;
    const int64_t tot = cum[units], all = tot * a.HK, per = stretch(a, all);
    const int64_t w = blockIdx.x;
    int64_t x = w * per;
    const int64_t xe = min(x + per, all);
    while (x < xe) {
        const int kvh = (int)(x / tot);
        const int64_t y = x - kvh * tot;
        const int u = find_unit(cum, units, y);
        const Unit un = unit_of(a, prefix, u);
        const int inside = (int)(y - cum[u]), rb = inside / un.tiles, first = inside % un.tiles;
        const int count = (int)min((int64_t)(un.tiles - first), xe - x);
        const bool whole = count == un.tiles;

        // the lane's row
        const int r = rb * 32 * RW + 32 * rw + (lane & 31);
        const bool real = r < un.rows;
        const int rc = min(r, un.rows - 1), token = un.tok0 + rc / a.per, head = kvh * a.per + rc % a.per;
        int seq = u;
        if (prefix) seq = a.cu ? find_seq(a.cu, a.N, token) : token;
        const int ctx = a.context[seq];
        const int seen = ctx < 0 ? 0 : (int)min((int64_t)ctx + (token - seq_first(a, seq)) + 1, (int64_t)un.key1);
        typename C::Q q;
        C::load_q(static_cast<const char*>(a.q) + ((int64_t)token * a.q_stride + (int64_t)head * D) * L::es, half, a.negate, q);
        AttnRow<T, D> acc;
        const int32_t* const table = a.table + (int64_t)un.table * a.max_pages;

        for (int ti = first; ti < first + count; ++ti) {
            const int j0 = un.key0 + ti * kKeys;
            auto at = [&](const void* pages, int row) {
                const int j = min(j0 + row, un.key1 - 1);
                int p = table[j >> a.page_shift];
                p = p >= 0 && p < a.num_pages ? p : 0;
                return static_cast<const char*>(pages) +
                       ((((int64_t)p * a.HK + kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * L::row_bytes;
            };
            constexpr int per = L::template per<kKeys, WAVES>();
#pragma unroll
            for (int i = 0; i < per; ++i) {
                const int f = 64 * (per * wave + i), row = L::copy_row(f, lane);
                const char* kp = at(a.k_pages, row) + L::template copy_byte<false>(f, lane);
                const char* vp = at(a.v_pages, row) + L::template copy_byte<true>(f, lane);
                asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(kp), "s"(sk + 16 * f) : "memory");
                asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(vp), "s"(sv + 16 * f) : "memory");
            }
            wait_copies();
            __syncthreads();
            f32x16_t s[blocks];
#pragma unroll
            for (int b = 0; b < blocks; ++b) {
                const int block = KW == 2 ? kw : b;
                s[b] = C::scores(block, at_, q);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int j16 = j0 + 32 * block + 16 * g;
                    const int p = j16 < un.key1 ? table[j16 >> a.page_shift] : -1;
                    const int lim = p >= 0 && p < a.num_pages ? seen : 0;
#pragma unroll
                    for (int i = 8 * g; i < 8 * g + 8; ++i)
                        s[b][i] = j0 + 32 * block + key_of(i, half) < lim ? s[b][i] : kNegInf;
                }
            }
            acc.add(s, a.c, KW == 2 ? kw : 0, at_);
            __syncthreads();
        }
        float l = both_sum(acc.l), m = acc.m;
        f32x16_t* const o = acc.o;
        if constexpr (KW == 2) {   // the two waves of a row block: the odd one's part joins the even one's
            float* const mine = xch + rw * 64 * 18 + lane;
            if (kw == 1) { mine[16 * 64] = m; mine[17 * 64] = l; }
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                if (kw == 1)
#pragma unroll
                    for (int i = 0; i < 16; ++i) mine[i * 64] = o[b][i];
                __syncthreads();
                if (kw == 0) {
                    const float m1 = mine[16 * 64], l1 = mine[17 * 64], mn = fmaxf(m, m1);
                    const float base = mn == kNegInf ? 0.0f : mn * a.c;
                    const float e0 = __builtin_amdgcn_exp2f(m * a.c - base), e1 = __builtin_amdgcn_exp2f(m1 * a.c - base);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[b][i] = o[b][i] * e0 + mine[i * 64] * e1;
                    if (b == D / 32 - 1) { l = l * e0 + l1 * e1; m = mn; }
                }
                __syncthreads();
            }
        }
        if (kw == 0) {
            if (whole && !a.groups) {
                const bool store = real && ctx >= 0;
                const float inv = reciprocal_sum(l);
                char* row = store ? static_cast<char*>(a.o) + ((int64_t)token * a.HQ + head) * L::row_bytes : nullptr;
#pragma unroll
                for (int b = 0; b < D / 32; ++b) o[b] *= inv;
                C::store(row, half, o);
                if (a.lse && store && half == 0)
                    a.lse[(int64_t)token * a.HQ + head] = log_sum(m * a.c, l);
            } else if (real) {
                const int64_t slot = whole ? 2 * (int64_t)a.workers + (int64_t)kvh * item[units] + item[u] + rb : open_slot(w, first > 0);
                float* s = reinterpret_cast<float*>(slots + slot * slot_bytes);
                const int row = 32 * rw + (lane & 31);
                C::store_part(s + row * D, half, o);
                if (half == 0) {
                    s[32 * RW * D + row] = m == kNegInf ? kNegInf : m * a.c;
                    s[32 * RW * D + 32 * RW + row] = l;
                }
            }
        }
        x += count;
    }
}

// One wave per (token, query head): its parts joined.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnPagedArgs a) {
    constexpr int V = D / 64;
    const int lane = threadIdx.x & 63;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (id >= a.T * a.HQ) return;
    const int token = (int)(id / a.HQ), head = (int)(id % a.HQ);
    if (a.cu && token >= a.cu[a.N]) return;
    const int seq = a.cu ? find_seq(a.cu, a.N, token) : token;
    if (a.context[seq] < 0) return;
    const int kvh = head / a.per, hh = head % a.per;
    float m = kNegInf, l = 0.0f, o[V] = {};
    bool written = false;
    for (int side = 0; side < 2; ++side) {
        const bool prefix = side == 1;
        const int u = prefix ? a.group[seq] : seq;
        if (u < 0) continue;
        const Unit un = unit_of(a, prefix, u);
        if (un.tiles <= 0) continue;
        const int64_t* cum = prefix ? a.prefix_cum : a.cum;
        const int* item = prefix ? a.prefix_item : a.item;
        const int units = prefix ? a.groups : a.N, rows = prefix ? a.prefix_rows : a.rows;
        const char* slots = prefix ? a.prefix_slots : a.slots;
        const int64_t slot_bytes = (int64_t)rows * (D + 2) * 4, tot = cum[units], per = stretch(a, tot * a.HK);
        const int r = (token - un.tok0) * a.per + hh, rb = r / rows, row = r % rows;
        const int64_t x0 = kvh * tot + cum[u] + (int64_t)rb * un.tiles, x1 = x0 + un.tiles;
        const int64_t w0 = x0 / per, w1 = (x1 - 1) / per;
        if (w0 == w1 && !a.groups) { written = true; break; }
        for (int64_t w = w0; w <= w1; ++w) {
            const int64_t slot = w0 == w1 ? 2 * (int64_t)a.workers + (int64_t)kvh * item[units] + item[u] + rb : open_slot(w, w > w0);
            const float* s = reinterpret_cast<const float*>(slots + slot * slot_bytes);
            const float m1 = s[rows * D + row], l1 = s[rows * D + rows + row];
            const float mn = fmaxf(m, m1), base = mn == kNegInf ? 0.0f : mn;
            const float e0 = __builtin_amdgcn_exp2f(m - base), e1 = __builtin_amdgcn_exp2f(m1 - base);
            m = mn;
            l = l * e0 + l1 * e1;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = o[i] * e0 + s[row * D + V * lane + i] * e1;
        }
    }
    if (written) return;
    const float inv = reciprocal_sum(l);
#pragma unroll
    for (int i = 0; i < V; ++i) Elem<T>::store(a.o, id * D + V * lane + i, o[i] * inv);
    if (a.lse && lane == 0) a.lse[id] = log_sum(m, l);
}

template <typename T, int D>
hipError_t launch_part(const AttnPagedArgs& a, int rows, bool prefix, hipStream_t stream) {
    const dim3 grid((unsigned)a.workers);
    if (rows == 32) attn_paged_kernel<T, D, 2, 1><<<grid, 128, 0, stream>>>(a, prefix);
    else if (rows == 64) attn_paged_kernel<T, D, 2, 2><<<grid, 256, 0, stream>>>(a, prefix);
    else attn_paged_kernel<T, D, 1, 4><<<grid, 256, 0, stream>>>(a, prefix);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch(const AttnPagedArgs& a, hipStream_t stream) {
    attn_plan_kernel<<<1, 1024, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.groups) e = launch_part<T, D>(a, a.prefix_rows, true, stream);
    if (e == hipSuccess) e = launch_part<T, D>(a, a.rows, false, stream);
    if (e != hipSuccess) return e;
    attn_join_kernel<T, D><<<dim3((unsigned)((a.T * a.HQ + 3) / 4)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

int rows_for(int64_t rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

AttnPagedPlan attn_paged_plan(int64_t T, int32_t N, int32_t HQ, int32_t HK, int D, int32_t max_q_len, int32_t groups) {
    AttnPagedPlan p{};
    const int64_t per = HQ / HK;
    p.workers = 512;
    p.rows = rows_for(per * max_q_len);
    p.prefix_rows = rows_for(per * T);
    auto slots = [&](int rows, int64_t units) {
        // two open parts per workgroup; with prefixes nothing is written straight to the output
        int64_t n = 2 * p.workers;
        if (groups) n += (units + (T * per + rows - 1) / rows) * HK;
        return up((size_t)n * rows * (D + 2) * 4);
    };
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t r = at; at += up(bytes); return r; };
    p.cum = take((size_t)(N + 1) * 8);
    p.item = take((size_t)(N + 1) * 4);
    p.pre = take((size_t)N * 4);
    p.group = take((size_t)N * 4);
    p.prefix_cum = take((size_t)(groups + 1) * 8);
    p.prefix_item = take((size_t)(groups + 1) * 4);
    p.prefix = take((size_t)groups * 4);
    p.rep = take((size_t)groups * 4);
    p.slots = take(slots(p.rows, N));
    p.prefix_slots = groups ? take(slots(p.prefix_rows, groups)) : at;
    p.total = at;
    return p;
}

hipError_t launch_attn_paged(AttnPagedArgs a, const AttnPagedPlan& p, char* ws, int D, int io_dtype, hipStream_t stream) {
    a.workers = p.workers; a.rows = p.rows; a.prefix_rows = p.prefix_rows;
    a.per = a.HQ / a.HK;
    a.capacity = (int64_t)a.max_pages << a.page_shift;
    a.cum = reinterpret_cast<int64_t*>(ws + p.cum);
    a.item = reinterpret_cast<int32_t*>(ws + p.item);
    a.pre = reinterpret_cast<int32_t*>(ws + p.pre);
    a.group = reinterpret_cast<int32_t*>(ws + p.group);
    a.prefix_cum = reinterpret_cast<int64_t*>(ws + p.prefix_cum);
    a.prefix_item = reinterpret_cast<int32_t*>(ws + p.prefix_item);
    a.prefix = reinterpret_cast<int32_t*>(ws + p.prefix);
    a.rep = reinterpret_cast<int32_t*>(ws + p.rep);
    a.slots = ws + p.slots;
    a.prefix_slots = ws + p.prefix_slots;
    if (io_dtype == 1) return D == 64 ? launch<bf16_t, 64>(a, stream) : launch<bf16_t, 128>(a, stream);
    return D == 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace gdr
