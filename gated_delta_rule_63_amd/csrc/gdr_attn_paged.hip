// Attention of a few tokens per sequence against a paged cache, with prefixes that groups of sequences share
// (gdr_attn_decode_paged).
//
// The tokens of one sequence (or, over a shared prefix, of a whole group) times the query heads of one key head
// are the rows of one product: keys and values are read once for all of them.  The work of a key head is a line of
// tiles of 64 keys, (unit, row block, tile) in that order, cut into equal stretches for a fixed number of
// workgroups, whatever the lengths are: the host does not know them, and every workgroup sums them up for itself.
// A stretch may end inside a unit; such a part's maximum, sum and unnormalised output go to the workspace and are
// joined by the last kernel.
//   attn_paged_kernel   the groups' prefixes (with prefixes), then what is each sequence's own
//   attn_join_kernel    parts -> outputs
//
// Long caches are bound by HBM: 64 sequences of up to 8191 tokens, 8 key heads of 128 bf16 channels, 976 MB, take 175 us
// (5.6 TB/s) and their join 5; 1..12 tokens each against up to 4095, 554 MB, 124 + 9.  Short ones are bound by latency:
// one sequence of 4097 tokens (17 MB) takes 12.0 + 5.2 us, a chain of dependent loads (lengths, page, tile) and two tiles;
// stretches of at least two or four tiles took as long or 1.5 us longer.  With a prefix of 16384 tokens for 64 sequences
// its parts are a third of the traffic: 33 us (17% of the matrix unit's cycles), then 25 for up to 512 own tokens each and
// 10 to join.  32 x 8 fp32 beams over 1000 tokens with up to 127 of their own: 24 + 28 + 6 us, the matrix unit busy 22% and
// 15%; 4 rows fill an eighth of a block, whose products are a chain of their own in each wave, behind the start and the first
// tile.  fp32 rows of 128 channels in blocks of 64 and 128 (q_len 12: 64 sequences against up to 4095 tokens 344 us of a
// floor of 224) keep 18 and 16 registers in scratch memory; no other kernel does.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "gdr_attn_device.h"

namespace gdr {
namespace {

constexpr int kKeys = 64;       // keys per tile
constexpr int kJoinGroups = 1 << 16;   // workgroups that join with prefixes, at most (a launch has fewer than 2^32 threads)

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

// tiles of a stretch, of a line of so many
__device__ __forceinline__ int stretch(const AttnPagedArgs& a, int tiles) {
    return max((int)(((int64_t)tiles + a.per_head - 1) / a.per_head), 1);
}

// Group g's sequences [s, e), the first of them that is not padded (its pages are the group's; -1: none) and the keys in
// whole pages of the prefix.
struct Group { int s, e, rep, prefix; };
__device__ __forceinline__ int group_offset(const AttnPagedArgs& a, int i) { return max(0, min(a.group_offsets[i], a.N)); }
__device__ __forceinline__ Group group_of(const AttnPagedArgs& a, int g) {
    Group r;
    r.s = group_offset(a, g);
    r.e = max(r.s, group_offset(a, g + 1));
    r.rep = -1;
    for (int n = r.s; n < r.e && r.rep < 0; ++n)
        if (keys_of(a, a.context[n], a.cu ? a.cu[n + 1] - a.cu[n] : 1) > 0) r.rep = n;
    const int64_t len = r.rep < 0 ? 0 : min((int64_t)max(0, a.prefix_lens[g]), a.capacity);
    r.prefix = (int)(len >> a.page_shift << a.page_shift);
    return r;
}

// Each sequence's group and the keys that it reads with it, for the kernels behind this one: workgroup by workgroup.
__device__ __forceinline__ void tell_groups(const AttnPagedArgs& a) {
    for (int g = blockIdx.x; g < a.groups; g += gridDim.x) {
        const Group x = group_of(a, g);
        for (int n = x.s + threadIdx.x; n < x.e; n += blockDim.x) { a.pre[n] = x.prefix; a.group[n] = g; }
        if (threadIdx.x == 0) { a.prefix[g] = x.prefix; a.first[g] = x.s; }
    }
    if (blockIdx.x == 0) {   // the sequences of none
        const int s = group_offset(a, 0), e = group_offset(a, a.groups);
        if (threadIdx.x == 0) a.first[a.groups] = e;
        for (int n = threadIdx.x; n < a.N; n += blockDim.x)
            if (n < s || n >= e) { a.pre[n] = 0; a.group[n] = -1; }
    }
}

struct Unit {
    int tok0, rows;      // first token, tokens * heads per key head
    int key0, key1;      // keys
    int table;           // row of the page table
    int tiles, blocks;   // tiles of keys, blocks of rows; both 0 if there are no keys
};

template <bool PREFIX>
__device__ __forceinline__ Unit unit_of(const AttnPagedArgs& a, int u, int block_rows) {
    Unit r;
    if (PREFIX) {
        const Group g = group_of(a, u);
        r.key0 = 0;
        r.key1 = g.prefix;
        r.tok0 = seq_first(a, g.s);
        r.rows = (seq_first(a, g.e) - r.tok0) * a.per;
        r.table = g.rep;
    } else {
        const int ctx = a.context[u];
        r.key0 = a.groups ? a.pre[u] : 0;
        r.tok0 = seq_first(a, u);
        const int tokens = seq_first(a, u + 1) - r.tok0;
        r.rows = tokens * a.per;
        r.key1 = keys_of(a, ctx, tokens);
        r.table = u;
    }
    const bool some = r.key1 > r.key0 && r.rows > 0;
    r.tiles = some ? (r.key1 - r.key0 + kKeys - 1) / kKeys : 0;
    r.blocks = some ? (r.rows + block_rows - 1) / block_rows : 0;
    return r;
}

// The line of tiles of one key head (below 2^31: the host sees to it): sums before every THREADS-th part of the units,
// in the LDS.
template <int THREADS> struct Line {
    int tiles[THREADS + 1];
    int items[THREADS + 1];      // row blocks
    int wave_tiles[THREADS / 64], wave_items[THREADS / 64];
};

// units: of THREADS units at most, what they are, for find_items
template <bool PREFIX, int THREADS>
__device__ __forceinline__ void sum_up(const AttnPagedArgs& a, int units, int block_rows, Line<THREADS>& line, Unit* cache) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int run = (units + THREADS - 1) / THREADS, u0 = min(tid * run, units), u1 = min(u0 + run, units);
    int t = 0, n = 0;
    Unit x{};
    for (int u = u0; u < u1; ++u) {
        x = unit_of<PREFIX>(a, u, block_rows);
        t += x.tiles * x.blocks;
        n += x.blocks;
    }
    cache[tid] = x;
    int tiles = wave_scan(t), items = wave_scan(n);
    if (lane == 63) { line.wave_tiles[wave] = tiles; line.wave_items[wave] = items; }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w)
        if (w < wave) { tiles += line.wave_tiles[w]; items += line.wave_items[w]; }
    line.tiles[tid] = tiles - t;   // before the thread's units
    line.items[tid] = items - n;
    if (tid == THREADS - 1) { line.tiles[THREADS] = tiles; line.items[THREADS] = items; }
    __syncthreads();
}

// the unit that tile y of the line is in, and the tiles and row blocks before it
template <bool PREFIX, int THREADS>
__device__ __forceinline__ int find_unit(const AttnPagedArgs& a, int units, int block_rows, const Line<THREADS>& line, int y,
                                         int& tiles, int& items) {
    const int lane = threadIdx.x & 63, run = (units + THREADS - 1) / THREADS;
    int part = -1;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) part += __popcll(__ballot(line.tiles[64 * i + lane] <= y));
    int t0 = uniform(line.tiles[part]), n0 = uniform(line.items[part]), u = part * run;
    for (int u0 = part * run; run > 1; u0 += 64) {
        Unit x{};
        if (u0 + lane < min((part + 1) * run, units)) x = unit_of<PREFIX>(a, u0 + lane, block_rows);
        const int mine = x.tiles * x.blocks, t = wave_scan(mine), n = wave_scan(x.blocks);
        const uint64_t here = __ballot(t0 + t - mine <= y && y < t0 + t);
        if (here || u0 + 64 >= (part + 1) * run) {   // the second never without the first
            const int k = here ? __builtin_ctzll(here) : 63;
            t0 += lane_value(t - mine, k);
            n0 += lane_value(n - x.blocks, k);
            u = u0 + k;
            break;
        }
        t0 += lane_value(t, 63);
        n0 += lane_value(n, 63);
    }
    tiles = t0;
    items = n0;
    return u;
}

// The maximum of a part that saw scores of -inf only: above that of one that saw nothing, below all that have a sum.
constexpr float kLost = -__FLT_MAX__;

// Parts of a unit's row block: the slots they are in.  Workgroup w has one for a block that it goes on with and one for a
// block that it leaves unfinished; where outputs are joined anyway, a block that it holds whole has one of its own.
__device__ __forceinline__ int64_t open_slot(int64_t w, bool continued) { return 2 * w + (continued ? 0 : 1); }

// A place on the line: tiles [tile, tile + count) of a unit's row block.
struct Item {
    int token0, row0, rows;    // the unit's first token; the block's first row and the unit's rows
    int key0, key1;            // the unit's keys
    int table;                 // row of the page table
    int tile, count, tiles;
    int item;                  // row blocks before it on the line of a key head
    int unit;
};
constexpr int kItems = 64;     // found at a time

// The items of tiles [y, ye) of key head kvh's line, kItems of them at most, by one wave: 64 units at a time.  `next` is
// where the rest begins.
template <bool PREFIX, int THREADS>
__device__ __forceinline__ int find_items(const AttnPagedArgs& a, int units, int block_rows, const Line<THREADS>& line,
                                          const Unit* cache, int kvh, int y, int ye, Item* items, int& next, int32_t* starts,
                                          int32_t* item_starts) {
    const int lane = threadIdx.x & 63;
    int t0, n0;
    const int u = find_unit<PREFIX>(a, units, block_rows, line, y, t0, n0) + lane;
    Unit un{};
    if (u < units) un = cache ? cache[u] : unit_of<PREFIX>(a, u, block_rows);
    const int mine = un.tiles * un.blocks;
    const int behind = t0 + wave_scan(mine), t = behind - mine;   // behind and before the lane's unit
    const int n = n0 + wave_scan(un.blocks) - un.blocks;
    const int a0 = max(t, y), a1 = min(behind, ye);               // the unit's tiles in the stretch
    const int rb0 = a0 < a1 ? (a0 - t) / un.tiles : 0, rb1 = a0 < a1 ? (a1 - t - 1) / un.tiles : -1;
    const int count = rb1 - rb0 + 1, upto = wave_scan(count), at = upto - count, all = lane_value(upto, 63);
    if (count > 0) {
        for (int rb = rb0; rb <= rb1 && at + rb - rb0 < kItems; ++rb) {
            const int r = t + rb * un.tiles;
            Item it;
            it.token0 = un.tok0; it.row0 = rb * block_rows; it.rows = un.rows;
            it.key0 = un.key0; it.key1 = un.key1; it.table = un.table;
            it.tile = max(r, y) - r;
            it.count = min(r + un.tiles, ye) - r - it.tile;
            it.tiles = un.tiles; it.item = n + rb;
            it.unit = u;
            items[at + rb - rb0] = it;
        }
        // whoever begins a unit tells the last kernel where it is on the line
        if (kvh == 0 && t >= y) { starts[u] = t; item_starts[u] = n; }
    }
    // behind the last unit looked at, or the first item that there was no room for
    int end = min(ye, lane_value(behind, 63));
    if (all > kItems) {
        const uint64_t who = __ballot(count > 0 && at <= kItems && upto > kItems);
        end = lane_value(t + (rb0 + kItems - at) * un.tiles, __builtin_ctzll(who));
    }
    next = end;
    return min(all, kItems);
}

// an item that every lane holds alike, in scalar registers
__device__ __forceinline__ Item same(const Item& it) {
    Item r;
    r.token0 = uniform(it.token0); r.row0 = uniform(it.row0); r.rows = uniform(it.rows);
    r.key0 = uniform(it.key0); r.key1 = uniform(it.key1); r.table = uniform(it.table);
    r.tile = uniform(it.tile); r.count = uniform(it.count); r.tiles = uniform(it.tiles);
    r.item = uniform(it.item); r.unit = uniform(it.unit);
    return r;
}

template <typename T, int D, int KW, int RW, bool PREFIX>
__global__ __launch_bounds__(64 * KW * RW, 2) void attn_paged_kernel(AttnPagedArgs a) {
    using L = AttnTile<T, D>;
    using C = AttnCore<T, D>;
    constexpr int WAVES = KW * RW, THREADS = 64 * WAVES, blocks = 2 / KW, block_rows = 32 * RW;
    constexpr int tile_bytes = kKeys * L::row_bytes;
    // Two tiles of fp32 rows of 128 channels would leave room for one workgroup on a CU.  With one, the next keys are on their way
    // during the softmax and the products with the values, the next values during the products with the keys (64 sequences of
    // up to 8191 tokens 360 us, with two tiles 631).
    constexpr bool ONE = L::row_bytes == 512;
    __shared__ __align__(1024) char lds[(ONE ? 2 : 4) * tile_bytes];
    __shared__ float xch[RW][2][64];
    __shared__ Line<THREADS> line;
    __shared__ Item items[kItems];
    __shared__ int found, rest;
    __shared__ uint32_t special_rows[2][kKeys / 32];

    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), half = lane >> 5;
    const int kw = wave % KW, rw = wave / KW;
    const int units = PREFIX ? a.groups : a.N;
    char* const slots = PREFIX ? a.prefix_slots : a.slots;
    int32_t* const starts = PREFIX ? a.prefix_start : a.start;
    int32_t* const item_starts = PREFIX ? a.prefix_item : a.item;
    constexpr int64_t slot_bytes = (int64_t)block_rows * (D + 2) * 4;
    const int w = blockIdx.x, kvh = w / a.per_head;
    if (threadIdx.x < 4) special_rows[threadIdx.x >> 1][threadIdx.x & 1] = 0;
    int turn = 0;

    Unit* cache = reinterpret_cast<Unit*>(lds);   // of the first items; the tiles come over it
    static_assert(THREADS * sizeof(Unit) <= sizeof(lds), "units in the tiles' place");
    sum_up<PREFIX>(a, units, block_rows, line, cache);
    if (units > THREADS) cache = nullptr;
    if (w == 0 && threadIdx.x == 0) { starts[units] = line.tiles[THREADS]; item_starts[units] = line.items[THREADS]; }
    if (!PREFIX && threadIdx.x == 0) a.open[w].parts = 0;
    if (PREFIX) tell_groups(a);

    // pages of a tile's four runs of 16 keys; -1: none
    struct Pages { int p[4]; };
    auto pages_of = [&](int row, int j0, int key1) {
        const int32_t* const table = a.table + (int64_t)row * a.max_pages;
        int p[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) p[g] = uniform_load(table + (min(j0 + 16 * g, key1 - 1) >> a.page_shift));
        Pages r;
#pragma unroll
        for (int g = 0; g < 4; ++g) r.p[g] = j0 + 16 * g < key1 && p[g] >= 0 && p[g] < a.num_pages ? p[g] : -1;
        return r;
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
    auto stage_part = [&](const Pages& pages, int j0, int key1, uint32_t to, auto keys, auto values) {
#pragma unroll
        for (int g = 0; g < groups16; ++g) {
            const int r0 = 16 * (groups16 * wave + g), j = j0 + r0, last = key1 - 1 - j;
            int p = pages.p[g];
            if constexpr (WAVES == 2) p = wave ? pages.p[2 + g] : p;
            else p = wave == 0 ? p : wave == 1 ? pages.p[1] : wave == 2 ? pages.p[2] : pages.p[3];
            const int64_t off = ((((int64_t)p * a.HK + kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * L::row_bytes;
            const char* const k = copy_base(p >= 0 ? static_cast<const char*>(a.k_pages) + off : zero_rows);
            const char* const v = copy_base(p >= 0 ? static_cast<const char*>(a.v_pages) + off : zero_rows);
            const uint32_t dst = to + r0 * L::row_bytes;
            if (last >= 15 || p < 0) {
#pragma unroll
                for (int i = 0; i < copies; ++i) {
                    if constexpr (keys.value) copy_to_lds(k, ko[i], dst + 1024 * i);
                    if constexpr (values.value) copy_to_lds(v, vo[i], dst + tile_bytes + 1024 * i);
                }
            } else {   // behind the last key, which nobody sees: that key again, and zeros for values (0 * inf)
                typedef __attribute__((address_space(3))) f32x4_t lds_f4;
#pragma unroll
                for (int i = 0; i < copies; ++i) {
                    const int over = max(L::copy_row(64 * i, lane) - last, 0);
                    if constexpr (keys.value) copy_to_lds(k, ko[i] - over * L::row_bytes, dst + 1024 * i);
                    if constexpr (values.value) {
                        if (over > 0) *(lds_f4*)(uintptr_t)(dst + tile_bytes + 1024 * i + 16 * lane) = f32x4_t{};
                        else copy_to_lds(v, vo[i], dst + tile_bytes + 1024 * i);
                    }
                }
            }
        }
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    auto stage = [&](const Pages& pages, int j0, int key1, uint32_t to) { stage_part(pages, j0, key1, to, yes, yes); };

    uint32_t to = base;
    typename C::At at(base, base + tile_bytes, lane);
    const int tot = uniform(line.tiles[THREADS]), per = stretch(a, tot), part = w % a.per_head;
    // (in 64 bits: stretches behind the line's end)
    const int ye = (int)min(((int64_t)part + 1) * per, (int64_t)tot);
    for (int y = (int)min((int64_t)part * per, (int64_t)tot), y_next; y < ye; y = y_next) {
        if (wave == 0) {
            int next;
            const int n = find_items<PREFIX>(a, units, block_rows, line, cache, kvh, y, ye, items, next, starts, item_starts);
            if (lane == 0) { found = n; rest = next; }
        }
        cache = nullptr;
        __syncthreads();
        // into registers before the barrier below: behind it the first wave goes on and writes them again
        const int n_items = uniform(found);
        y_next = uniform(rest);
        if constexpr (!ONE) {
            const Item it = same(items[0]);
            const int j0 = it.key0 + it.tile * kKeys;
            stage(pages_of(it.table, j0, it.key1), j0, it.key1, to);
        }
        for (int i = 0; i < n_items; ++i) {
            const Item it = same(items[i]), next = same(items[min(i + 1, n_items - 1)]);
            const bool more = i + 1 < n_items;
            Pages now = pages_of(it.table, it.key0 + it.tile * kKeys, it.key1);
            if constexpr (ONE) {
                const int j0 = it.key0 + it.tile * kKeys;
                stage_part(now, j0, it.key1, to, yes, no);
                stage_part(now, j0, it.key1, to, no, yes);
            }
            // the lane's row
            const int r = it.row0 + 32 * rw + (lane & 31);
            const bool real = r < it.rows;
            const int rc = min(r, it.rows - 1), token = it.token0 + rc / a.per, head = kvh * a.per + rc % a.per;
            const int seq = !PREFIX ? it.unit : a.cu ? find_seq(a.cu, a.N, token) : token;
            const int ctx = a.context[seq];
            const int seen = ctx < 0 ? 0 : (int)min((int64_t)ctx + (token - seq_first(a, seq)) + 1, (int64_t)it.key1);
            typename C::Q q;
            C::load_q(static_cast<const char*>(a.q) + ((int64_t)token * a.q_stride + (int64_t)head * D) * L::es, half, a.negate, q);
            AttnRow<T, D> acc;
            const int end = it.tile + it.count;
            for (int tile = it.tile; tile < end; ++tile) {
                // the next tile's pages, read while this one's copies are waited for
                const bool inside = tile + 1 < end;
                const int key1 = inside ? it.key1 : next.key1;
                const int ahead0 = inside ? it.key0 + (tile + 1) * kKeys : next.key0 + next.tile * kKeys;
                const Pages ahead = pages_of(inside ? it.table : next.table, ahead0, key1);
                f32x16_t s[blocks];
                if constexpr (ONE) {
                    // the values' copies are the last ones (fewer of them where rows behind the last key take zeros)
                    if (it.key0 + (tile + 1) * kKeys <= it.key1) wait_copies<copies * groups16>();
                    else wait_copies();
                    __syncthreads();
#pragma unroll
                    for (int b = 0; b < blocks; ++b) s[b] = C::scores(KW == 2 ? kw : b, at, q);
                }
                wait_copies();
                __syncthreads();
                const uint32_t v = to + tile_bytes;
                if constexpr (ONE) {
                    if (inside) stage_part(ahead, ahead0, key1, to, yes, no);
                } else {
                    to = 2 * base + 2 * tile_bytes - to;
                    if (inside || more) stage(ahead, ahead0, key1, to);
                }

                const int j0 = it.key0 + tile * kKeys;
                // tokens see less than the last of theirs: some rows do not see what others do
                const bool uneven = !PREFIX && it.rows > a.per && j0 + kKeys > it.key1 - it.rows / a.per + 1;
                if (uneven) {
                    turn ^= 1;
                    take_out_specials<T, D, kKeys, WAVES>(v, special_rows, turn, wave, lane);
                }
                if constexpr (!ONE)
#pragma unroll
                    for (int b = 0; b < blocks; ++b) s[b] = C::scores(KW == 2 ? kw : b, at, q);
                int pages = 0;   // bit g: keys 16 g .. 16 g + 15 of the tile are in the cache
#pragma unroll
                for (int g = 0; g < 4; ++g) pages |= (now.p[g] >= 0) << g;
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
                if (uneven)
                    for (int b = 0; b < blocks; ++b)
                        for (uint32_t left = uniform((int)special_rows[turn][blocks * kw + b]); left; left &= left - 1) {
                            const int k = 32 * (blocks * kw + b) + __builtin_ctz(left), j = j0 + k;
                            const int p = k < 16 ? now.p[0] : k < 32 ? now.p[1] : k < 48 ? now.p[2] : now.p[3];
                            if (j < seen && p >= 0)
                                C::add_specials(static_cast<const char*>(a.v_pages) +
                                                ((((int64_t)p * a.HK + kvh) << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * L::row_bytes,
                                                half, acc.o);
                        }
                if constexpr (ONE) {
                    __syncthreads();
                    if (inside) stage_part(ahead, ahead0, key1, to, no, yes);
                } else {
                    at.move(to == base ? (uint32_t)(-2 * tile_bytes) : 2 * tile_bytes);
                }
                now = ahead;
            }

            const bool whole = it.count == it.tiles;
            float l = both_sum(acc.l), m = acc.m;
            f32x16_t* const o = acc.o;
            if constexpr (KW == 2) {   // the two waves of a row block
                // in the place of the last tile, which the next copies do not touch before the next barrier
                static_assert(RW * 64 * D / 2 * 4 <= 2 * tile_bytes, "outputs in a tile's place");
                float* const place = reinterpret_cast<float*>(lds + (ONE ? 0 : 2 * tile_bytes - (to - base))) + rw * (64 * D / 2);
                join_waves<D, KW>(o, m, l, a.c, place, &xch[rw][0][0], kw, lane);
            }
            if (kw == 0) {
                // No weight at all: nothing that is in the cache, or scores of -inf only.  Looked up for those rows alone, so that the
                // loop over the tiles carries nothing for it.
                bool lost = false;
                if (__any(real && l == 0.0f)) {
                    const Item x = same(items[i]);
                    const int left = l == 0.0f ? seen : 0;
                    for (int tile = x.tile; tile < x.tile + x.count; ++tile) {
                        const int j0 = x.key0 + tile * kKeys;
                        if (!__any(left > j0)) break;
                        const Pages p = pages_of(x.table, j0, x.key1);
#pragma unroll
                        for (int g = 0; g < 4; ++g) lost |= p.p[g] >= 0 && left - j0 > 16 * g;
                    }
                }
                if (whole && !a.groups) {
                    const bool store = real && ctx >= 0;
                    if (lost) l = no_sum();
                    const float inv = reciprocal_sum(l);
                    char* row = store ? static_cast<char*>(a.o) + ((int64_t)token * a.HQ + head) * L::row_bytes : nullptr;
#pragma unroll
                    for (int b = 0; b < D / 32; ++b) o[b] *= inv;
                    C::store(row, half, o);
                    if (a.lse && store && half == 0) a.lse[(int64_t)token * a.HQ + head] = log_sum(m * a.c, l);
                } else if (real) {
                    const int64_t slot = whole ? 2 * (int64_t)a.workers + (int64_t)kvh * line.items[THREADS] + it.item : open_slot(w, it.tile > 0);
                    float* s = reinterpret_cast<float*>(slots + slot * slot_bytes);
                    const int row = 32 * rw + (lane & 31);
                    C::store_part(s + row * D, half, o);
                    if (half == 0) {
                        s[block_rows * D + row] = lost ? kLost : m;
                        s[block_rows * D + block_rows + row] = l;
                    }
                }
            }
            // the block that it leaves unfinished, for the last kernel
            const int left = it.tiles - it.count;
            if constexpr (ONE) __syncthreads();   // the next item's copies come over the parts
            if (!PREFIX && it.tile == 0 && left > 0 && threadIdx.x == 0)
                a.open[w] = AttnOpen{it.token0, it.row0, min(block_rows, it.rows - it.row0), kvh, 1 + (left + per - 1) / per};
        }
        __syncthreads();   // before the next items are found
    }
}

// A part of a row: its output in the slot and, `stats` and `stats + rows` floats behind, its maximum and its sum.
struct Part { const float* row; int stats, rows; };
template <int D> __device__ __forceinline__ Part part_at(const char* slots, int64_t slot, int rows, int row) {
    return {reinterpret_cast<const float*>(slots + slot * ((int64_t)rows * (D + 2) * 4)) + row * D, rows * D + row - row * D, rows};
}

// Parts of a row, joined by LANES = 32 or 64 lanes: a lane reads the maximum and the sum of one part, then each half of
// the wave reads the rows, all of them or every second one.
template <typename T, int D, int LANES, typename F>
__device__ __forceinline__ void join_row(const AttnPagedArgs& a, int token, int head, int parts, F part_of) {
    constexpr int V = D / 32, turns = LANES / 32;
    typedef float vec_t __attribute__((ext_vector_type(V)));
    const int part = threadIdx.x & (LANES - 1), lane = threadIdx.x & 31, turn = part >> 5;
    float m = kNegInf, l = 0.0f;
    vec_t o = {};
    for (int k0 = 0; k0 < parts; k0 += LANES) {
        const int n = min(LANES, parts - k0);
        float m1 = kNegInf, l1 = 0.0f;
        if (part < n) {
            const Part p = part_of(k0 + part);
            m1 = p.row[p.stats];
            l1 = p.row[p.stats + p.rows];
        }
        float mn = m1;
#pragma unroll
        for (int d = 1; d < LANES; d *= 2) mn = fmaxf(mn, __shfl_xor(mn, d));
        mn = fmaxf(mn, m);
        const float base = mn == kNegInf ? 0.0f : mn;
        const float e = __builtin_amdgcn_exp2f((m1 - base) * a.c), e0 = __builtin_amdgcn_exp2f((m - base) * a.c);
        l1 *= e;
#pragma unroll
        for (int d = 1; d < LANES; d *= 2) l1 += __shfl_xor(l1, d);
        m = mn;
        l = l * e0 + l1;
        o *= e0;
        constexpr int ahead = 8;
        for (int p = 0; p < n; p += ahead * turns) {
            vec_t y[ahead];
            float f[ahead];
#pragma unroll
            for (int q = 0; q < ahead; ++q) {
                const int k = p + turns * q + turn, kk = min(k, n - 1);
                f[q] = __shfl(e, kk, LANES);
                y[q] = reinterpret_cast<const vec_t*>(part_of(k0 + kk).row)[lane];
            }
#pragma unroll
            for (int q = 0; q < ahead; ++q)
                if (p + turns * q + turn < n) o += y[q] * f[q];   // (a value may be infinite: not by a weight of 0)
        }
    }
    if constexpr (turns == 2)
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] += __shfl_xor(o[i], 32);
    if (turn > 0) return;
    if (l == 0.0f && m > kNegInf) l = no_sum();
    const int64_t id = (int64_t)token * a.HQ + head;
    const float inv = reciprocal_sum(l);
    if constexpr (Elem<T>::bytes == 4) {
        reinterpret_cast<vec_t*>(static_cast<float*>(a.o) + id * D)[lane] = o * inv;
    } else {
        uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + id * D) + lane * (V / 2);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) to[i] = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
    }
    if (a.lse && lane == 0) a.lse[id] = log_sum(m * a.c, l);
}

// Without prefixes: LANES lanes for every row of the blocks that stretches have left unfinished; and the rows that see
// nothing although their sequence is not padded (a table without room), which no tile belongs to.
template <typename T, int D, int LANES>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnPagedArgs a) {
    constexpr int rows = 256 / LANES;
    const int w = blockIdx.x, mine = blockIdx.y * rows + threadIdx.x / LANES;
    if (w < a.workers) {
        const AttnOpen x = a.open[w];
        const int r = mine;
        if (r >= x.rows || x.parts == 0) return;
        const int row = x.row0 + r;
        join_row<T, D, LANES>(a, x.token0 + row / a.per, x.kvh * a.per + row % a.per, x.parts,
                       [&](int k) { return part_at<D>(a.slots, open_slot(w + k, k > 0), a.rows, r); });
        return;
    }
    const int64_t all = rows * (int64_t)gridDim.y, step = all * (gridDim.x - a.workers);
    for (int64_t id = (w - a.workers) * all + mine; id < a.T * a.HQ; id += step) {
        const int token = (int)(id / a.HQ);
        if ((a.cu && token >= a.cu[a.N]) || a.context[a.cu ? find_seq(a.cu, a.N, token) : token] < 0) continue;
        join_row<T, D, LANES>(a, token, (int)(id % a.HQ), 0, [](int) { return Part{}; });
    }
}

// With prefixes: LANES lanes per (token, query head); parts of the prefix and of the sequence's own keys.
template <typename T, int D, int LANES>
__global__ __launch_bounds__(256) void attn_join_groups_kernel(AttnPagedArgs a) {
    constexpr int rows = 256 / LANES;
    for (int64_t id = (int64_t)blockIdx.x * rows + threadIdx.x / LANES; id < a.T * a.HQ; id += rows * (int64_t)gridDim.x) {
        const int token = (int)(id / a.HQ), head = (int)(id % a.HQ);
        if (a.cu && token >= a.cu[a.N]) return;
        const int seq = a.cu ? find_seq(a.cu, a.N, token) : token;
        // all that depends on the sequence, then all that depends on its group (what an empty unit has not been told is not used)
        const Unit un = unit_of<false>(a, seq, a.rows);
        const int ctx = a.context[seq], group = a.group[seq], own_start = a.start[seq], own_item = a.item[seq];
        const int own_tiles = a.start[a.N], own_items = a.item[a.N], pre_tiles = a.prefix_start[a.groups], pre_items = a.prefix_item[a.groups];
        const int g = max(group, 0), pre_keys = a.prefix[g], pre_tok0 = seq_first(a, a.first[g]), pre_start = a.prefix_start[g], pre_item = a.prefix_item[g];
        if (ctx < 0) continue;
        const int kvh = head / a.per, hh = head % a.per;
        struct Side { int64_t first, own; int parts, row; };
        auto side = [&](int tok0, int tiles, int rows, int start, int item, int all_tiles, int all_items) {
            const int per = stretch(a, all_tiles), r = (token - tok0) * a.per + hh, rb = r / rows;
            const int x0 = start + rb * tiles, w0 = x0 / per, w1 = (x0 + tiles - 1) / per;
            return Side{(int64_t)kvh * a.per_head + w0, 2 * (int64_t)a.workers + (int64_t)kvh * all_items + item + rb, w1 - w0 + 1, r % rows};
        };
        const Side own = un.tiles > 0 ? side(un.tok0, un.tiles, a.rows, own_start, own_item, own_tiles, own_items) : Side{0, 0, 0, 0};
        const Side pre = group >= 0 && pre_keys > 0
            ? side(pre_tok0, (pre_keys + kKeys - 1) / kKeys, a.prefix_rows, pre_start, pre_item, pre_tiles, pre_items) : Side{0, 0, 0, 0};
        join_row<T, D, LANES>(a, token, head, pre.parts + own.parts, [&](int k) {
            const bool p = k < pre.parts;
            const Side s = p ? pre : own;
            const int i = p ? k : k - pre.parts;
            return part_at<D>(p ? a.prefix_slots : a.slots, s.parts == 1 ? s.own : open_slot(s.first + i, i > 0), p ? a.prefix_rows : a.rows, s.row);
        });
    }
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
    if (a.groups) e = launch_part<T, D, true>(a, a.prefix_rows, stream);
    if (e == hipSuccess) e = launch_part<T, D, false>(a, a.rows, stream);
    if (e != hipSuccess) return e;
    if (a.groups) {
        // half a wave for each of many rows: 64 heads, 182 sequences of up to 5 tokens 69 us for all kernels (with a wave 95), 32 x 8
        // fp32 beams of 16 heads 56 (57); a wave for few: 64 tokens, 32 heads, 33 parts 65 (67)
        if (a.T * a.HQ < 4096) attn_join_groups_kernel<T, D, 64><<<dim3((unsigned)((a.T * a.HQ + 3) / 4)), 256, 0, stream>>>(a);
        else attn_join_groups_kernel<T, D, 32><<<dim3((unsigned)min((a.T * a.HQ + 7) / 8, (int64_t)kJoinGroups)), 256, 0, stream>>>(a);
    } else {
        // few rows are likely to have many parts (one sequence of 4097 tokens, 33 parts: 6.0 us with a wave per row, 7.4 with
        // half a one), many rows few (64 sequences of 1..12 tokens, 2 or 3 parts of 48 rows: 12.4 and 9.3)
        const unsigned across = (unsigned)(a.workers + (a.capacity == 0 ? 256 : 0));
        if (a.rows == 32) attn_join_kernel<T, D, 64><<<dim3(across, 8), 256, 0, stream>>>(a);
        else attn_join_kernel<T, D, 32><<<dim3(across, (unsigned)(a.rows / 8)), 256, 0, stream>>>(a);
    }
    return hipGetLastError();
}

int rows_for(int64_t rows) { return rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

AttnPagedPlan attn_paged_plan(int64_t T, int32_t N, int32_t HQ, int32_t HK, int D, int32_t max_q_len, int32_t groups) {
    AttnPagedPlan p{};
    const int64_t per = HQ / HK;
    // as many as are resident at once, by their LDS; each has one key head
    p.per_head = max(1, 512 / HK);
    p.workers = p.per_head * HK;
    p.rows = rows_for(per * max_q_len);
    p.prefix_rows = groups ? rows_for((per * T + groups - 1) / groups) : 0;   // of a group of average size
    auto slots = [&](int rows, int64_t units) {
        // two open parts per workgroup; with prefixes nothing is written straight to the output
        int64_t n = 2 * (int64_t)p.workers;
        if (groups) n += (units + (T * per + rows - 1) / rows) * HK;
        return up((size_t)n * rows * (D + 2) * 4);
    };
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t r = at; at += up(bytes); return r; };
    p.start = take((size_t)(N + 1) * 4);
    p.item = take((size_t)(N + 1) * 4);
    if (groups) {
        p.pre = take((size_t)N * 4);
        p.group = take((size_t)N * 4);
        p.prefix_start = take((size_t)(groups + 1) * 4);
        p.prefix_item = take((size_t)(groups + 1) * 4);
        p.prefix = take((size_t)groups * 4);
        p.first = take((size_t)(groups + 1) * 4);
        p.prefix_slots = take(slots(p.prefix_rows, groups));
    }
    p.open = take((size_t)p.workers * sizeof(AttnOpen));
    p.slots = take(slots(p.rows, N));
    p.total = at;
    return p;
}

hipError_t launch_attn_paged(AttnPagedArgs a, const AttnPagedPlan& p, char* ws, int D, int io_dtype, hipStream_t stream) {
    a.workers = p.workers; a.per_head = p.per_head; a.rows = p.rows; a.prefix_rows = p.prefix_rows;
    a.per = a.HQ / a.HK;
    a.capacity = (int64_t)a.max_pages << a.page_shift;
    a.start = reinterpret_cast<int32_t*>(ws + p.start);
    a.item = reinterpret_cast<int32_t*>(ws + p.item);
    a.pre = reinterpret_cast<int32_t*>(ws + p.pre);
    a.group = reinterpret_cast<int32_t*>(ws + p.group);
    a.prefix_start = reinterpret_cast<int32_t*>(ws + p.prefix_start);
    a.prefix_item = reinterpret_cast<int32_t*>(ws + p.prefix_item);
    a.prefix = reinterpret_cast<int32_t*>(ws + p.prefix);
    a.first = reinterpret_cast<int32_t*>(ws + p.first);
    a.open = reinterpret_cast<AttnOpen*>(ws + p.open);
    a.slots = ws + p.slots;
    a.prefix_slots = ws + p.prefix_slots;
    if (io_dtype == 1) return D == 64 ? launch<bf16_t, 64>(a, stream) : launch<bf16_t, 128>(a, stream);
    return D == 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace gdr
