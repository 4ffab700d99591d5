// Attention of a few tokens per sequence against a paged cache, with prefixes that groups of sequences share
// (gdr_attn_decode_paged).
//
// The tokens of one sequence (or, over a shared prefix, of a whole group) times the query heads of one key head
// are the rows of one product: keys and values are read once for all of them.  The work is a line of tiles of 64
// keys, (key head, unit, row block, tile) in that order, cut into equal stretches for a fixed number of
// workgroups, whatever the lengths are: the host does not know them, and every workgroup sums them up for itself.
// A stretch may end inside a unit; such a part's maximum, sum and unnormalised output go to the workspace and are
// joined by the last kernel.
//   attn_groups_kernel  (with prefixes) each group's pages and length, each sequence's group
//   attn_paged_kernel   the groups' prefixes, then what is each sequence's own
//   attn_join_kernel    parts -> outputs
#include <hip/hip_runtime.h>

#include "gdr_attn_device.h"

namespace gdr {
namespace {

constexpr int kKeys = 64;       // keys per tile
constexpr int kMinTiles = 2;    // tiles of a workgroup's stretch at least: below, parts cost more than they save

// what stands for a page outside the cache: finite rows that nobody sees
__device__ __align__(256) const char zero_rows[16 * 512] = {};

// A value that is the same in every lane, read through the scalar cache: apart from the copies in flight, whose wait
// is that of the vector loads.  Only for what this launch does not write.
__device__ __forceinline__ int uniform_load(const int32_t* p) {
    return *(__attribute__((address_space(4))) const int32_t*)(uintptr_t)p;
}

__device__ __forceinline__ int seq_first(const AttnPagedArgs& a, int n) { return a.cu ? a.cu[n] : n; }

// keys that a sequence's last token sees; 0 for a padded sequence and one without tokens
__device__ __forceinline__ int keys_of(const AttnPagedArgs& a, int ctx, int tokens) {
    return ctx < 0 || tokens <= 0 ? 0 : (int)min((int64_t)ctx + tokens, a.capacity);
}

__device__ __forceinline__ int64_t stretch(const AttnPagedArgs& a, int64_t tiles) {
    return max((tiles + a.workers - 1) / a.workers, (int64_t)kMinTiles);
}

// One wave per group: the first sequence that is not padded gives the pages, whole pages are shared.  The wave behind
// the last group takes the sequences of none.
__global__ __launch_bounds__(256) void attn_groups_kernel(AttnPagedArgs a) {
    const int lane = threadIdx.x & 63, g = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (g > a.groups) return;
    auto offset = [&](int i) { return max(0, min(a.group_offsets[i], a.N)); };
    if (g == a.groups) {
        const int s = offset(0), e = offset(a.groups);
        for (int n = lane; n < a.N; n += 64)
            if (n < s || n >= e) { a.pre[n] = 0; a.group[n] = -1; }
        return;
    }
    const int s = offset(g), e = max(s, offset(g + 1));
    int rep = -1;
    for (int n0 = s; n0 < e && rep < 0; n0 += 64) {
        const int n = n0 + lane;
        const bool live = n < e && keys_of(a, a.context[n], a.cu ? a.cu[n + 1] - a.cu[n] : 1) > 0;
        const uint64_t some = __ballot(live);
        if (some) rep = n0 + __builtin_ctzll(some);
    }
    const int64_t len = rep < 0 ? 0 : min((int64_t)max(0, a.prefix_lens[g]), a.capacity);
    const int pre = (int)(len >> a.page_shift << a.page_shift);
    for (int n = s + lane; n < e; n += 64) { a.pre[n] = pre; a.group[n] = g; }
    if (lane == 0) {
        a.rep[g] = rep;
        a.prefix[g] = pre;
        a.first[g] = s;
        if (g == a.groups - 1) a.first[a.groups] = e;
    }
}

struct Unit {
    int tok0, rows;      // first token, tokens * heads per key head
    int key0, key1;      // keys
    int tiles, blocks;   // tiles of keys, blocks of rows; both 0 if there are no keys
};

template <bool PREFIX>
__device__ __forceinline__ Unit unit_of(const AttnPagedArgs& a, int u, int block_rows) {
    Unit r;
    if (PREFIX) {
        const int s = a.first[u], e = a.first[u + 1];
        r.tok0 = seq_first(a, s);
        r.rows = (seq_first(a, e) - r.tok0) * a.per;
        r.key0 = 0;
        r.key1 = a.prefix[u];
    } else {
        r.tok0 = seq_first(a, u);
        const int tokens = seq_first(a, u + 1) - r.tok0;
        r.rows = tokens * a.per;
        r.key0 = a.groups ? a.pre[u] : 0;
        r.key1 = keys_of(a, a.context[u], tokens);
    }
    const bool some = r.key1 > r.key0 && r.rows > 0;
    r.tiles = some ? (r.key1 - r.key0 + kKeys - 1) / kKeys : 0;
    r.blocks = some ? (r.rows + block_rows - 1) / block_rows : 0;
    return r;
}

// The line of tiles of one key head: sums before every THREADS-th part of the units, in the LDS.
template <int THREADS> struct Line {
    int64_t tiles[THREADS + 1];
    int items[THREADS + 1];      // row blocks
    int64_t wave_tiles[THREADS / 64];
    int wave_items[THREADS / 64];
};

template <bool PREFIX, int THREADS>
__device__ __forceinline__ void sum_up(const AttnPagedArgs& a, int units, int block_rows, Line<THREADS>& line) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int run = (units + THREADS - 1) / THREADS, u0 = min(tid * run, units), u1 = min(u0 + run, units);
    int64_t t = 0;
    int n = 0;
    for (int u = u0; u < u1; ++u) {
        const Unit x = unit_of<PREFIX>(a, u, block_rows);
        t += (int64_t)x.tiles * x.blocks;
        n += x.blocks;
    }
    const int64_t mine = t;
    const int mine_n = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t tt = __shfl_up(t, d);
        const int nn = __shfl_up(n, d);
        if (lane >= d) { t += tt; n += nn; }
    }
    if (lane == 63) { line.wave_tiles[wave] = t; line.wave_items[wave] = n; }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w)
        if (w < wave) { t += line.wave_tiles[w]; n += line.wave_items[w]; }
    line.tiles[tid] = t - mine;
    line.items[tid] = n - mine_n;
    if (tid == THREADS - 1) { line.tiles[THREADS] = t; line.items[THREADS] = n; }
    __syncthreads();
}

// the unit that tile y of the line is in, and the tiles and row blocks before it
template <bool PREFIX, int THREADS>
__device__ __forceinline__ int find_unit(const AttnPagedArgs& a, int units, int block_rows, const Line<THREADS>& line, int64_t y,
                                         int64_t& tiles, int& items) {
    const int lane = threadIdx.x & 63, run = (units + THREADS - 1) / THREADS;
    int part = -1;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) part += __popcll(__ballot(line.tiles[64 * i + lane] <= y));
    part = __builtin_amdgcn_readfirstlane(part);
    int64_t t0 = line.tiles[part];
    int n0 = line.items[part], u = part * run;
    for (int u0 = part * run; run > 1; u0 += 64) {
        Unit x{};
        if (u0 + lane < min((part + 1) * run, units)) x = unit_of<PREFIX>(a, u0 + lane, block_rows);
        const int64_t mine = (int64_t)x.tiles * x.blocks;
        int64_t t = mine;
        int n = x.blocks;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int64_t tt = __shfl_up(t, d);
            const int nn = __shfl_up(n, d);
            if (lane >= d) { t += tt; n += nn; }
        }
        const uint64_t here = __ballot(t0 + t - mine <= y && y < t0 + t);
        const int k = here ? __builtin_ctzll(here) : 63;
        const int64_t before = t0 + __shfl(t, k) - __shfl(mine, k);
        const int before_n = n0 + __shfl(n, k) - __shfl(x.blocks, k);
        if (here || u0 + 64 >= (part + 1) * run) {   // the second never without the first
            t0 = before; n0 = before_n; u = u0 + k;
            break;
        }
        t0 += __shfl(t, 63); n0 += __shfl(n, 63);
    }
    tiles = t0;
    items = n0;
    return __builtin_amdgcn_readfirstlane(u);
}

// Parts of a unit's row block: the slots they are in.  Workgroup w has one for a block that it goes on with and one for a
// block that it leaves unfinished; where outputs are joined anyway, a block that it holds whole has one of its own.
__device__ __forceinline__ int64_t open_slot(int64_t w, bool continued) { return 2 * w + (continued ? 0 : 1); }

// A place on the line: row block `rb` of unit `u` for key head `kvh`, tiles [tile, tile + count) of it.
struct Item {
    Unit un;
    int kvh, u, rb, tile, count, items;
    int64_t tiles;
};

template <typename T, int D, int KW, int RW, bool PREFIX>
__global__ __launch_bounds__(64 * KW * RW) void attn_paged_kernel(AttnPagedArgs a) {
    using L = AttnTile<T, D>;
    using C = AttnCore<T, D>;
    constexpr int WAVES = KW * RW, THREADS = 64 * WAVES, blocks = 2 / KW, block_rows = 32 * RW;
    constexpr int tile_bytes = kKeys * L::row_bytes;
    __shared__ __align__(1024) char lds[4 * tile_bytes];
    __shared__ float xch[KW == 2 ? RW * 64 * 18 : 1];
    __shared__ Line<THREADS> line;
    __shared__ uint32_t special_rows[2][2];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    const int kw = wave % KW, rw = wave / KW;
    const int units = PREFIX ? a.groups : a.N;
    char* const slots = PREFIX ? a.prefix_slots : a.slots;
    int64_t* const starts = PREFIX ? a.prefix_start : a.start;
    int32_t* const item_starts = PREFIX ? a.prefix_item : a.item;
    constexpr int64_t slot_bytes = (int64_t)block_rows * (D + 2) * 4;
    const int64_t w = blockIdx.x;
    if (threadIdx.x < 4) special_rows[threadIdx.x >> 1][threadIdx.x & 1] = 0;
    int turn = 0;

    sum_up<PREFIX>(a, units, block_rows, line);
    const int64_t tot = line.tiles[THREADS], all = tot * a.HK, per = stretch(a, all);
    const int all_items = line.items[THREADS];
    if (w == 0 && threadIdx.x == 0) { starts[units] = tot; item_starts[units] = all_items; }
    int64_t x = w * per;
    const int64_t xe = min(x + per, all);
    if (x >= xe) return;

    auto item_at = [&](int64_t x) {
        Item it;
        it.kvh = (int)(x / tot);
        const int64_t y = x - it.kvh * tot;
        it.u = find_unit<PREFIX>(a, units, block_rows, line, y, it.tiles, it.items);
        it.un = unit_of<PREFIX>(a, it.u, block_rows);
        const int inside = (int)(y - it.tiles);
        it.rb = __builtin_amdgcn_readfirstlane(inside / it.un.tiles);
        it.tile = __builtin_amdgcn_readfirstlane(inside % it.un.tiles);
        it.count = (int)min((int64_t)(it.un.tiles - it.tile), xe - x);
        it.un.key0 = __builtin_amdgcn_readfirstlane(it.un.key0);
        it.un.key1 = __builtin_amdgcn_readfirstlane(it.un.key1);
        it.kvh = __builtin_amdgcn_readfirstlane(it.kvh);
        return it;
    };
    auto table_of = [&](const Item& it) {
        const int n = PREFIX ? __builtin_amdgcn_readfirstlane(a.rep[it.u]) : it.u;
        return a.table + (int64_t)n * a.max_pages;
    };
    auto page_at = [&](const int32_t* table, int j) {
        const int p = uniform_load(table + (j >> a.page_shift));
        return p >= 0 && p < a.num_pages ? p : -1;
    };

    // the lane's places in the copies of 16 rows
    constexpr int copies = L::template per<16, 1>(), groups16 = 4 / WAVES;
    uint32_t ko[copies], vo[copies];
#pragma unroll
    for (int i = 0; i < copies; ++i) {
        const int row = L::copy_row(64 * i, lane) * L::row_bytes;
        ko[i] = row + L::template copy_byte<false>(64 * i, lane);
        vo[i] = row + L::template copy_byte<true>(64 * i, lane);
    }
    const uint32_t base = lds_address(lds);
    auto stage = [&](const Item& it, const int32_t* table, int tile, uint32_t to) {
#pragma unroll
        for (int g = 0; g < groups16; ++g) {
            const int r0 = 16 * (groups16 * wave + g), j = it.un.key0 + tile * kKeys + r0, last = it.un.key1 - 1 - j;
            const int p = last >= 0 ? page_at(table, j) : -1;
            const int64_t off = ((((int64_t)p * a.HK + it.kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * L::row_bytes;
            const char* const k = p >= 0 ? static_cast<const char*>(a.k_pages) + off : zero_rows;
            const char* const v = p >= 0 ? static_cast<const char*>(a.v_pages) + off : zero_rows;
            const uint32_t dst = to + r0 * L::row_bytes;
            if (last >= 15 || p < 0) {
#pragma unroll
                for (int i = 0; i < copies; ++i) {
                    copy_to_lds(k, ko[i], dst + 1024 * i);
                    copy_to_lds(v, vo[i], dst + tile_bytes + 1024 * i);
                }
            } else {   // rows behind the last key stand for it
#pragma unroll
                for (int i = 0; i < copies; ++i) {
                    const uint32_t over = max(L::copy_row(64 * i, lane) - last, 0) * L::row_bytes;
                    copy_to_lds(k, ko[i] - over, dst + 1024 * i);
                    copy_to_lds(v, vo[i] - over, dst + tile_bytes + 1024 * i);
                }
            }
        }
    };

    Item it = item_at(x);
    const int32_t* table = table_of(it);
    uint32_t to = base;
    stage(it, table, it.tile, to);
    typename C::At at(base, base + tile_bytes, lane);
    while (true) {
        // the lane's row
        const int r = it.rb * block_rows + 32 * rw + (lane & 31);
        const bool real = r < it.un.rows;
        const int rc = min(r, it.un.rows - 1), token = it.un.tok0 + rc / a.per, head = it.kvh * a.per + rc % a.per;
        const int seq = !PREFIX ? it.u : a.cu ? find_seq(a.cu, a.N, token) : token;
        const int ctx = a.context[seq];
        const int seen = ctx < 0 ? 0 : (int)min((int64_t)ctx + (token - seq_first(a, seq)) + 1, (int64_t)it.un.key1);
        typename C::Q q;
        C::load_q(static_cast<const char*>(a.q) + ((int64_t)token * a.q_stride + (int64_t)head * D) * L::es, half, a.negate, q);
        AttnRow<T, D> acc;
        x += it.count;
        const bool more = x < xe;
        Item next;
        const int32_t* next_table = nullptr;
        if (more) {
            next = item_at(x);
            next_table = table_of(next);
        }
        const int end = it.tile + it.count;
        for (int tile = it.tile; tile < end; ++tile) {
            wait_copies();
            __syncthreads();
            const uint32_t v = to + tile_bytes;
            to = 2 * base + 2 * tile_bytes - to;
            if (tile + 1 < end) stage(it, table, tile + 1, to);
            else if (more) stage(next, next_table, next.tile, to);

            const int j0 = it.un.key0 + tile * kKeys;
            // tokens see less than the last of theirs: some rows do not see what others do
            uint64_t special = 0;
            if (!PREFIX && it.un.rows > a.per && j0 + kKeys > it.un.key1 - it.un.rows / a.per + 1) {
                special = take_out_specials<T, D, kKeys, WAVES>(v, special_rows, turn, wave, lane);
                turn ^= 1;
            }
            f32x16_t s[blocks];
#pragma unroll
            for (int b = 0; b < blocks; ++b) s[b] = C::scores(KW == 2 ? kw : b, at, q);
            int pages = 0;   // bit g: keys 16 g .. 16 g + 15 of the tile are in the cache
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (j0 + 16 * g < it.un.key1 && page_at(table, j0 + 16 * g) >= 0) pages |= 1 << g;
            if (pages != 15 || !__all(seen >= j0 + kKeys)) {
#pragma unroll
                for (int b = 0; b < blocks; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int k = 32 * (KW == 2 ? kw : b) + key_of(i, half);
                        s[b][i] = j0 + k < seen && (pages >> (k >> 4) & 1) ? s[b][i] : kNegInf;
                    }
            }
            acc.add(s, a.c, KW == 2 ? kw : 0, at);
            for (; special; special &= special - 1) {
                const int k = __builtin_ctzll(special), j = j0 + k;
                if ((KW == 1 || k / 32 == kw) && j < seen) {
                    const int p = page_at(table, j);
                    if (p >= 0)
                        C::add_specials(static_cast<const char*>(a.v_pages) +
                                        ((((int64_t)p * a.HK + it.kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * L::row_bytes,
                                        half, acc.o);
                }
            }
            at.move(to == base ? (uint32_t)(-2 * tile_bytes) : 2 * tile_bytes);
        }

        const bool whole = it.count == it.un.tiles;
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
                    const float e0 = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((m - mn) * a.c);
                    const float e1 = m1 == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((m1 - mn) * a.c);
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
                if (a.lse && store && half == 0) a.lse[(int64_t)token * a.HQ + head] = log_sum(m * a.c, l);
            } else if (real) {
                const int64_t slot = whole ? 2 * (int64_t)a.workers + (int64_t)it.kvh * all_items + it.items + it.rb : open_slot(w, it.tile > 0);
                float* s = reinterpret_cast<float*>(slots + slot * slot_bytes);
                const int row = 32 * rw + (lane & 31);
                C::store_part(s + row * D, half, o);
                if (half == 0) {
                    s[block_rows * D + row] = m == kNegInf ? kNegInf : m * a.c;
                    s[block_rows * D + block_rows + row] = l;
                }
            }
        }
        // whoever begins a unit tells the last kernel where it is on the line
        if (it.kvh == 0 && it.rb == 0 && it.tile == 0 && threadIdx.x == 0) { starts[it.u] = it.tiles; item_starts[it.u] = it.items; }
        if (!more) break;
        it = next;
        table = next_table;
    }
}

// One wave per (token, query head): its parts joined.  A lane reads the maximum and the sum of one part, then all read
// the rows.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnPagedArgs a) {
    constexpr int V = D / 64;
    const int lane = threadIdx.x & 63;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (id >= a.T * a.HQ) return;
    const int token = __builtin_amdgcn_readfirstlane((int)(id / a.HQ)), head = __builtin_amdgcn_readfirstlane((int)(id % a.HQ));
    if (a.cu && token >= a.cu[a.N]) return;
    const int seq = a.cu ? find_seq(a.cu, a.N, token) : token;
    if (a.context[seq] < 0) return;
    const int kvh = head / a.per, hh = head % a.per;
    float m = kNegInf, l = 0.0f, o[V] = {};
    auto side = [&](const Unit& un, int u, int units, int rows, const int64_t* starts, const int32_t* items, const char* slots) {
        if (un.tiles <= 0) return true;
        const int64_t slot_bytes = (int64_t)rows * (D + 2) * 4, tot = starts[units], per = stretch(a, tot * a.HK);
        const int r = (token - un.tok0) * a.per + hh, rb = r / rows, row = r % rows;
        const int64_t x0 = kvh * tot + starts[u] + (int64_t)rb * un.tiles, w0 = x0 / per, w1 = (x0 + un.tiles - 1) / per;
        if (w0 == w1 && !a.groups) return false;   // written already
        for (int64_t wa = w0; wa <= w1; wa += 64) {
            const int n = (int)min((int64_t)64, w1 - wa + 1);
            int64_t at = 0;
            float m1 = kNegInf, l1 = 0.0f;
            if (lane < n) {
                const int64_t w = wa + lane;
                at = (w0 == w1 ? 2 * (int64_t)a.workers + (int64_t)kvh * items[units] + items[u] + rb : open_slot(w, w > w0)) * slot_bytes;
                const float* s = reinterpret_cast<const float*>(slots + at);
                m1 = s[rows * D + row];
                l1 = s[rows * D + rows + row];
            }
            float mn = m1;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) mn = fmaxf(mn, __shfl_xor(mn, d));
            mn = fmaxf(mn, m);
            const float base = mn == kNegInf ? 0.0f : mn;
            const float e = __builtin_amdgcn_exp2f(m1 - base), e0 = __builtin_amdgcn_exp2f(m - base);
            l1 *= e;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) l1 += __shfl_xor(l1, d);
            m = mn;
            l = l * e0 + l1;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] *= e0;
            constexpr int ahead = 8;
            for (int p = 0; p < n; p += ahead) {
                float y[ahead][V], f[ahead];
#pragma unroll
                for (int q = 0; q < ahead; ++q) {
                    const int k = min(p + q, n - 1);
                    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)at, k), hi = __builtin_amdgcn_readlane((uint32_t)(at >> 32), k);
                    const float* s = reinterpret_cast<const float*>(slots + ((int64_t)hi << 32 | lo)) + row * D + V * lane;
                    f[q] = p + q < n ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e), k)) : 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) y[q][i] = s[i];
                }
#pragma unroll
                for (int q = 0; q < ahead; ++q)
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] += p + q < n ? y[q][i] * f[q] : 0.0f;
            }
        }
        return true;
    };
    if (!side(unit_of<false>(a, seq, a.rows), seq, a.N, a.rows, a.start, a.item, a.slots)) return;
    if (a.groups && a.group[seq] >= 0)
        side(unit_of<true>(a, a.group[seq], a.prefix_rows), a.group[seq], a.groups, a.prefix_rows, a.prefix_start, a.prefix_item, a.prefix_slots);
    const float inv = reciprocal_sum(l);
#pragma unroll
    for (int i = 0; i < V; ++i) Elem<T>::store(a.o, id * D + V * lane + i, o[i] * inv);
    if (a.lse && lane == 0) a.lse[id] = log_sum(m, l);
}

template <typename T, int D, bool PREFIX>
hipError_t launch_part(const AttnPagedArgs& a, int rows, hipStream_t stream) {
    const dim3 grid((unsigned)a.workers);
    if (rows == 32) attn_paged_kernel<T, D, 2, 1, PREFIX><<<grid, 128, 0, stream>>>(a);
    else if (rows == 64) attn_paged_kernel<T, D, 2, 2, PREFIX><<<grid, 256, 0, stream>>>(a);
    else attn_paged_kernel<T, D, 1, 4, PREFIX><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch(const AttnPagedArgs& a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.groups) {
        attn_groups_kernel<<<dim3((unsigned)(a.groups / 4 + 1)), 256, 0, stream>>>(a);
        if ((e = hipGetLastError()) == hipSuccess) e = launch_part<T, D, true>(a, a.prefix_rows, stream);
    }
    if (e == hipSuccess) e = launch_part<T, D, false>(a, a.rows, stream);
    if (e != hipSuccess) return e;
    attn_join_kernel<T, D><<<dim3((unsigned)((a.T * a.HQ + 3) / 4)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

int rows_for(int64_t rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

AttnPagedPlan attn_paged_plan(int64_t T, int32_t N, int32_t HQ, int32_t HK, int D, int io_bytes, int32_t max_q_len, int32_t groups) {
    AttnPagedPlan p{};
    const int64_t per = HQ / HK;
    p.workers = D * io_bytes <= 256 ? 512 : 256;   // as many as are resident at once, by their LDS
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
    p.start = take((size_t)(N + 1) * 8);
    p.item = take((size_t)(N + 1) * 4);
    if (groups) {
        p.pre = take((size_t)N * 4);
        p.group = take((size_t)N * 4);
        p.prefix_start = take((size_t)(groups + 1) * 8);
        p.prefix_item = take((size_t)(groups + 1) * 4);
        p.prefix = take((size_t)groups * 4);
        p.rep = take((size_t)groups * 4);
        p.first = take((size_t)(groups + 1) * 4);
        p.prefix_slots = take(slots(p.prefix_rows, groups));
    }
    p.slots = take(slots(p.rows, N));
    p.total = at;
    return p;
}

hipError_t launch_attn_paged(AttnPagedArgs a, const AttnPagedPlan& p, char* ws, int D, int io_dtype, hipStream_t stream) {
    a.workers = p.workers; a.rows = p.rows; a.prefix_rows = p.prefix_rows;
    a.per = a.HQ / a.HK;
    a.capacity = (int64_t)a.max_pages << a.page_shift;
    a.start = reinterpret_cast<int64_t*>(ws + p.start);
    a.item = reinterpret_cast<int32_t*>(ws + p.item);
    a.pre = reinterpret_cast<int32_t*>(ws + p.pre);
    a.group = reinterpret_cast<int32_t*>(ws + p.group);
    a.prefix_start = reinterpret_cast<int64_t*>(ws + p.prefix_start);
    a.prefix_item = reinterpret_cast<int32_t*>(ws + p.prefix_item);
    a.prefix = reinterpret_cast<int32_t*>(ws + p.prefix);
    a.rep = reinterpret_cast<int32_t*>(ws + p.rep);
    a.first = reinterpret_cast<int32_t*>(ws + p.first);
    a.slots = ws + p.slots;
    a.prefix_slots = ws + p.prefix_slots;
    if (io_dtype == 1) return D == 64 ? launch<bf16_t, 64>(a, stream) : launch<bf16_t, 128>(a, stream);
    return D == 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace gdr
