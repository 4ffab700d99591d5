// Causal attention over packed prompts (gdr_attn_prefill_fwd).
//
// A workgroup owns 32 RW consecutive tokens of the packed batch and one query head: RW row blocks of 32 query rows, each
// a wave's, or KW waves' that share every tile's keys and join their parts at the end.
// Tiles of 32 to 128 keys and values go through the LDS once for all of them, copied a tile ahead.  Up to 64 sequences are cut
// into rows each for itself.  More are cut at fixed borders of the packed batch: a workgroup's rows may be several
// sequences', each row sees the tokens from its sequence's start to itself, and 128 one-token sequences are one
// workgroup's work.
//
// 16384 tokens of 32 heads of 128 channels, bf16, run 2199 GFLOP in 2.08 ms, 1059 TFLOP/s (a product of 8192 x 8192 x 8192 by
// the library 1139), with the matrix unit busy 55%, vector instructions 50% and the LDS 42% of the cycles at about 1.75 GHz: the
// softmax and the products take turns in a wave, and two waves to a SIMD hide a part of it.  8 ragged prompts, 32768 tokens
// together, 1.40 ms, 975 TFLOP/s (1.31 to 1.46 on other cards).  fp32 of 64 channels, 3 prompts, 3001 tokens together, 8 heads:
// 52 us, 81 of the 153 TFLOP/s of such a product, the matrix unit busy 49%; the longest row blocks decide.
#include <hip/hip_runtime.h>

#include "gdr_attn_device.h"

namespace gdr {
namespace {

constexpr int kSorted = 64;   // sequences, at most, whose tiles are sorted by cost

// keys of a tile
template <typename T, int D, int KW> constexpr int tile_keys() { return KW == 4 ? 128 : D * Elem<T>::bytes == 512 && KW == 1 ? 32 : 64; }

// ONE: the LDS holds one tile only, so that two workgroups fit a CU; the next keys are on their way during the softmax and the
// products with the values, the next values during the products with the keys.
template <typename T, int D, int KW, int RW, bool ONE>
__global__ __launch_bounds__(64 * KW * RW, 2) void attn_prefill_kernel(AttnPrefillArgs a) {
    using L = AttnTile<T, D>;
    using C = AttnCore<T, D>;
    constexpr int WAVES = KW * RW, kRows = 32 * RW;
    constexpr int kKeys = tile_keys<T, D, KW>(), blocks = kKeys / 32 / KW;
    constexpr int tile_bytes = kKeys * L::row_bytes;
    __shared__ __align__(1024) char lds[(ONE ? 2 : 4) * tile_bytes];
    __shared__ uint32_t special_rows[2][kKeys / 32];
    __shared__ float xch[RW * KW][64];
    if (threadIdx.x < kKeys / 16) special_rows[threadIdx.x / (kKeys / 32)][threadIdx.x % (kKeys / 32)] = 0;
    int turn = 0;

    int rank, head;
    {
        const int b = blockIdx.x;
        if (a.HQ % 8 == 0) {  // workgroups go round the eight XCDs: each keeps to its own heads' keys and values
            const int per = a.HQ / 8, x = b & 7, i = b >> 3;
            rank = i / per;
            head = x * per + i % per;
        } else {
            rank = b / a.HQ;
            head = b % a.HQ;
        }
    }
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), half = lane >> 5, kw = wave % KW, rw = wave / KW;
    const int end = a.cu ? uniform(a.cu[a.N]) : (int)a.T;
    // rows [t0, stop); `lo`: the first key that any of them sees; the lane's token t sees [start, t]
    int t0, stop, lo, start, latest;
    if (a.N <= kSorted) {
        // tiles are cut at the sequences' borders, the longest sequence first and its last tile first: what is begun last
        // is short, and neighbours share their keys and values in the L2 (3 prompts, 3001 fp32 tokens together: 81 us, at
        // fixed borders 107)
        const int first = lane < a.N && a.cu ? a.cu[lane] : 0, len = lane < a.N ? (a.cu ? a.cu[lane + 1] - first : (int)a.T) : 0;
        const int tiles = (len + kRows - 1) / kRows;
        int before = 0;   // tiles of the sequences ahead of the lane's
        for (int j = 0; j < a.N; ++j) {
            const int other = lane_value(len, j);
            before += other > len || (other == len && j < lane) ? (other + kRows - 1) / kRows : 0;
        }
        const uint64_t here = __ballot(before <= rank && rank < before + tiles);
        if (!here) return;
        const int n = __builtin_ctzll(here), p = lane_value(before + tiles - 1, n) - rank;
        lo = start = latest = lane_value(first, n);
        t0 = lo + p * kRows;
        stop = min(t0 + kRows, lo + lane_value(len, n));
    } else {
        // at fixed borders, the last first
        t0 = (a.tiles - 1 - rank) * kRows;
        if (t0 >= end) return;
        stop = min(t0 + kRows, end);
        lo = uniform(a.cu[find_seq(a.cu, a.N, t0)]);
        latest = uniform(a.cu[find_seq(a.cu, a.N, stop - 1)]);
        start = a.cu[find_seq(a.cu, a.N, min(t0 + 32 * rw + (lane & 31), stop - 1))];
    }
    const int t = t0 + 32 * rw + (lane & 31), tc = min(t, stop - 1), kvh = head / (a.HQ / a.HK);
    const int wlo = uniform(start), wfirst = t0 + 32 * rw, wlate = lane_value(start, 31);
    const int hi = stop, whi = min(wfirst + 32, stop);

    typename C::Q q;
    C::load_q(static_cast<const char*>(a.q) + ((int64_t)tc * a.q_stride + (int64_t)head * D) * L::es, half, a.negate, q);
    AttnRow<T, D> r;
    const char* const kb = static_cast<const char*>(a.k) + (int64_t)kvh * D * L::es;
    const char* const vb = static_cast<const char*>(a.v) + (int64_t)kvh * D * L::es;

    // the lane's places in a tile's copies; rows behind the last token stand for it (no row sees them)
    constexpr int per = L::template per<kKeys, WAVES>();
    const uint32_t ks = (uint32_t)a.k_stride * L::es, vs = (uint32_t)a.v_stride * L::es;
    uint32_t ko[per], vo[per];
    auto places = [&](int last) {
#pragma unroll
        for (int i = 0; i < per; ++i) {
            const int first = 64 * (per * wave + i), row = min(L::copy_row(first, lane), last);
            ko[i] = row * ks + L::template copy_byte<false>(first, lane);
            vo[i] = row * vs + L::template copy_byte<true>(first, lane);
        }
    };
    auto stage_keys = [&](int j0, uint32_t to) {
        if (j0 + kKeys > end) places(end - 1 - j0);
        const char* const k0 = copy_base(kb + (int64_t)j0 * a.k_stride * L::es);
#pragma unroll
        for (int i = 0; i < per; ++i) copy_to_lds(k0, ko[i], to + 1024 * (per * wave + i));
    };
    auto stage_values = [&](int j0, uint32_t to) {
        const char* const v0 = copy_base(vb + (int64_t)j0 * a.v_stride * L::es);
#pragma unroll
        for (int i = 0; i < per; ++i) copy_to_lds(v0, vo[i], to + tile_bytes + 1024 * (per * wave + i));
    };
    auto stage = [&](int j0, uint32_t to) { stage_keys(j0, to); stage_values(j0, to); };
    const uint32_t base = lds_address(lds);
    places(kKeys - 1);
    stage(lo, base);
    typename C::At at(base, base + tile_bytes, lane);
    uint32_t to = base + 2 * tile_bytes;
    for (int j0 = lo; j0 < hi; j0 += kKeys) {
        const bool next = j0 + kKeys < hi, here = j0 < whi && j0 + kKeys > wlo;
        f32x16_t s[blocks];
        if constexpr (ONE) {
            wait_copies<per>();   // the values' are behind the keys'
            __syncthreads();
            if (here)
#pragma unroll
                for (int b = 0; b < blocks; ++b) s[b] = C::scores(blocks * kw + b, at, q);
        }
        wait_copies();
        __syncthreads();
        if (next) {
            if constexpr (ONE) stage_keys(j0 + kKeys, base);
            else stage(j0 + kKeys, to);
        }
        const bool uneven = j0 + kKeys - 1 > t0 || j0 < latest;
        if (uneven) {
            turn ^= 1;
            take_out_specials<T, D, kKeys, WAVES>(ONE ? base + tile_bytes : 2 * base + 3 * tile_bytes - to, special_rows, turn, wave, lane);
        }
        if (here) {
            if constexpr (!ONE)
#pragma unroll
                for (int b = 0; b < blocks; ++b) s[b] = C::scores(blocks * kw + b, at, q);
            auto seen = [&](int j) { return j >= start && j <= t; };
            if (j0 + kKeys - 1 > wfirst || j0 < wlate)
#pragma unroll
                for (int b = 0; b < blocks; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[b][i] = seen(j0 + 32 * (blocks * kw + b) + key_of(i, half)) ? s[b][i] : kNegInf;
            r.add(s, a.c, blocks * kw, at);
            if (uneven)
                for (int b = 0; b < blocks; ++b)
                    for (uint32_t left = uniform((int)special_rows[turn][blocks * kw + b]); left; left &= left - 1) {
                        const int j = j0 + 32 * (blocks * kw + b) + __builtin_ctz(left);
                        if (seen(j) && j < stop) C::add_specials(vb + (int64_t)j * a.v_stride * L::es, half, r.o);
                    }
        }
        if constexpr (ONE) {
            __syncthreads();
            if (next) stage_values(j0 + kKeys, base);
        } else {
            const uint32_t by = to - base == 0 ? (uint32_t)(-2 * tile_bytes) : 2 * tile_bytes;
            at.move(by);
            to -= by;
        }
    }
    float l = both_sum(r.l);
    if constexpr (KW > 1) {
        static_assert(RW * KW * 64 * D <= (ONE ? 2 : 4) * tile_bytes, "outputs in the tiles' place");
        join_waves<D, KW>(r.o, r.m, l, a.c, reinterpret_cast<float*>(lds) + rw * (KW * 64 * D / 4), xch[rw * KW], kw, lane);
        if (kw > 0) return;
    }
    if (l == 0.0f) l = no_sum();   // a row sees itself at least
    const float inv = reciprocal_sum(l);
    char* row = t < stop ? static_cast<char*>(a.o) + ((int64_t)t * a.HQ + head) * L::row_bytes : nullptr;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) r.o[b] *= inv;
    C::store(row, half, r.o);
    if (a.lse && t < stop && half == 0) a.lse[(int64_t)t * a.HQ + head] = log_sum(r.m * a.c, l);
}

template <typename T, int D, int KW, int RW>
hipError_t start(AttnPrefillArgs a, hipStream_t stream) {
    a.tiles = (int)((a.T + 32 * RW - 1) / (32 * RW)) + (a.N <= kSorted ? a.N - 1 : 0);
    const int n = a.tiles * a.HQ;
    const auto run = [&](auto* kernel) {
        kernel<<<dim3((unsigned)n), 64 * KW * RW, 0, stream>>>(a);
        return hipGetLastError();
    };
    // Where two tiles leave room for one workgroup on a CU: with one tile each from nearly two rounds of the card on (fp32, 8
    // heads, 3 ragged prompts, tokens together: D = 64, 3001 tokens 53 us, with two tiles 69; 2500 tokens 46 and 57; D = 128,
    // 6000 tokens 345 and 392), and in less than one (bf16, 8 heads, D = 128, one prompt of 1000 tokens 17.5 and 19.8).  In
    // between two workgroups meet on some CUs while others are idle (fp32, D = 64, 1500 tokens of 3 prompts 31 and 28).
    // Two of D = 128 in fp32 and 128 keys do not fit at all.
    constexpr int two = 4 * tile_keys<T, D, KW>() * D * Elem<T>::bytes;
    if constexpr (two > 80 * 1024)
        if (two > 160 * 1024 || n <= 256 || n > 448) return run(attn_prefill_kernel<T, D, KW, RW, true>);
    if constexpr (two <= 160 * 1024) return run(attn_prefill_kernel<T, D, KW, RW, false>);
}

template <typename T, int D>
hipError_t launch(const AttnPrefillArgs& a, hipStream_t stream) {
    // `wide`: workgroups of 128 rows.  From 640 on they fill the card, and rows that share a tile's reads count most.  One prompt,
    // bf16: 32 heads, D = 128, 2000 tokens 53 us (56 in workgroups of 64 rows, by two waves each, which the rule takes: 512), 4000
    // 155 (180); 16 heads, D = 64, 6000 tokens 112 (118), 16000 580 (672).  Below, 64 rows: 32 heads, D = 128, 1000 tokens 25 us
    // (128 rows 28); 3 ragged prompts, fp32, 8 heads, D = 128, 6000 tokens together 350 (605), but 12000 1133 (1242, which the
    // rule takes).
    // Small batches of sequences that are long enough for four waves to share their keys take 32 rows by four waves (in brackets:
    // 64 rows).  bf16, 16 heads, one prompt: D = 64, 1000 tokens 13 us (16), 2000 27 (27); D = 128, 1000 tokens 19 (22), as 4
    // ragged prompts 14 (14), as 8 18 (12); 8 heads, one prompt of 3000 tokens 43 (54), yet 32 heads, 700 tokens 24 (20).
    // fp32, 8 heads, ragged prompts, tokens together: D = 64, 3 of 600 14 (19), 8 of 1000 18 (16), 16 of 3000 29 (27), 3 of 3001
    // 54 (89); D = 128, 3 of 1500 48 (69), 3 of 4000 204 (215); one head, one prompt of 1669 78 (121).
    const int64_t wide = (a.T + 127) / 128 * a.HQ;
    constexpr int es = Elem<T>::bytes, few = es == 4 ? 256 : 128, tokens = es == 4 ? 192 : 256;
    if (wide <= few && a.T >= (int64_t)tokens * a.N) return start<T, D, 4, 1>(a, stream);
    return wide < 640 ? start<T, D, 2, 2>(a, stream) : start<T, D, 1, 4>(a, stream);
}

}  // namespace

// of a large batch
int64_t attn_prefill_tiles(int64_t T) { return (T + 127) / 128 + kSorted; }

hipError_t launch_attn_prefill(AttnPrefillArgs a, int D, int io_dtype, hipStream_t stream) {
    if (io_dtype == 1) return D == 64 ? launch<bf16_t, 64>(a, stream) : launch<bf16_t, 128>(a, stream);
    return D == 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace gdr
