// Beam search for gfx950: the best candidates over beams and vocabulary, and the paged states moved to
// where the chosen beams expect them.
//
// Selection: s[w, v] = score[w] + logit[w, v] - log sum_v e^logit[w, v]; the best of the W V candidates
// of a batch row in descending order, equal ones by the lower beam, in a beam by the higher logit (different
// logits can give the same 64-bit score), then by the lower token.
//   rows   one workgroup per (row, part of the vocabulary), its logits in registers, read once: maximum,
//          sum of exponentials, and the part's best `out` entries by (logit, lower token).  Within a beam
//          the order of the candidates is the order of their logits, so these lists are exact.
//   merge  one workgroup per batch row: log-sum-exp per beam from the parts in 64 bits, scores of the
//          listed entries in 64 bits, the best `out` of them.  The sums come from 32-bit exponentials, so
//          scores of different beams closer than kNear could stand in the wrong order: where two
//          neighbours of the result are that close, or candidates behind it that close to its last one,
//          their beams' sums are formed again in 64 bits.
//
// Reordering: a parent's first child keeps its slot; the other children take, in order, the slots of
// parents without children, and only these are copied.  What is read (slots of parents with children) and
// what is written (slots of parents without) never meet, so all copies of all layers run at once.
#include "gdr_device.h"
#include "gdr_internal.h"

namespace gdr {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kWaveCap = 256;                      // entries above the threshold that a wave may list
constexpr int kWaveList = kWaveCap + kBeamMaxOut + 8;  // and those equal to it, and the padding to eight
constexpr int kMergeThreads = 256;
constexpr int kMaxSplits = 64;

// Bound of the difference between the 32-bit sums' log and the true one.  A logit's share passes four
// exponentials (about the thread's maximum, then the thread's, the wave's and the part's weight); each carries
// the hardware's 2^-23 and for a distance d its roundings (the difference, its product with log2 e, log2 e itself),
// 2.25 |d| 2^-24, and the four distances add up to the logit's distance to the row's maximum.  What lies beyond
// 20 is below 2^20 e^-20 = 2e-3 of the sum.  (4 + 22.5) 2^-23 = 3.2e-6, plus 3 additions in 32 bits (2e-7): two
// beams' scores are in the right order if they differ by more than twice 3.4e-6, and by what their own roundings
// to 64 bits come to beyond that: half a step, at most 2^-53 of the score, in each of the two and in each of
// the two that exact sums would give (2^-51, and as much again for the better one's step being the next larger).
constexpr double kNear = 7e-6;
__device__ __forceinline__ bool near_scores(double better, double worse) {
    return better - worse < fma(fabs(worse), 0x1p-50, kNear);
}

// Keys in ascending order of the float they stand for.  -0 counts as 0, NaN as -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.0f : -__builtin_inff(); }

__device__ __forceinline__ uint64_t entry_of(float x, uint32_t token) { return ((uint64_t)key_of(x) << 32) | ~token; }

// Reductions over the wave: four steps inside each row of 16 lanes by DPP, two across the rows.
__device__ __forceinline__ float row16_max(float x) {
    x = fmaxf(x, dpp_mov<0xB1>(x));
    x = fmaxf(x, dpp_mov<0x4E>(x));
    x = fmaxf(x, dpp_mov<0x141>(x));
    return fmaxf(x, dpp_mov<0x140>(x));
}
__device__ __forceinline__ float wave_max(float x) {
    x = row16_max(x);
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
template <int CTRL> __device__ __forceinline__ double dpp_mov64(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = __float_as_uint(dpp_mov<CTRL>(__uint_as_float((uint32_t)b)));
    const uint32_t hi = __float_as_uint(dpp_mov<CTRL>(__uint_as_float((uint32_t)(b >> 32))));
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double row16_sum64(double x) {
    x += dpp_mov64<0xB1>(x);
    x += dpp_mov64<0x4E>(x);
    x += dpp_mov64<0x141>(x);
    return x + dpp_mov64<0x140>(x);
}
__device__ __forceinline__ double wave_sum(double x) {
    x = row16_sum64(x);
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

__device__ __forceinline__ int lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Sorts n (a power of two) items of LDS, the first in order first; all threads of the workgroup call it.
template <int THREADS, typename Swap> __device__ __forceinline__ void bitonic_sort(int n, Swap swap_if_wrong) {
    for (int k = 2; k <= n; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            __syncthreads();
            for (int i = threadIdx.x; i < n / 2; i += THREADS) {
                const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1));
                swap_if_wrong(lo, lo | j, (lo & k) == 0);
            }
        }
    __syncthreads();
}

__device__ __forceinline__ int pow2_at_least(int n) { return n <= 2 ? 2 : 1 << (32 - __builtin_clz(n - 1)); }

template <int PER, bool CLEAN> __device__ __forceinline__ double sum_about(const float (&x)[PER], float about) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; i += 8) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = exp_f32((CLEAN ? clean(x[i + e]) : x[i + e]) - about);
        sum += (double)(((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7])));
    }
    return sum;
}

// PER logits per thread, in groups of eight that keep their maximum: most groups are never looked at again.
// VECW of a group at a time are neighbours (one aligned 16-byte load), or 1.  32 searches of 8 beams over 131072
// bf16 logits: 17.7 us (67 MB, 3.8 TB/s), VALU busy 42%; 4 beams over 32000: 5.4 us, a workgroup's latency.
template <typename IO, int PER, int VECW>
__global__ __launch_bounds__(kRowThreads, 4) void beam_rows_kernel(const BeamArgs a) {
    constexpr int G = PER / 8;
    const int row = blockIdx.y, split = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63;
    const int base = split * a.chunk;
    const int64_t row_at = (int64_t)row * a.stride;
    const float kNone = -__builtin_inff();

    __shared__ __align__(16) uint64_t list[kRowWaves][kWaveList];
    __shared__ double sh_sum[kRowWaves];
    __shared__ float sh_top[kRowWaves];
    __shared__ uint32_t sh_key[kRowThreads];
    __shared__ int listed[kRowWaves];

    const float score = a.scores[row];
    // ended beams and beams without probability list nothing
    if ((a.finished && a.finished[row]) || !(score > kNone && score < -kNone)) return;

    // element i of a thread: token base + token_of(i)
    uint32_t own = tid * VECW;
    auto token_of = [&](int i) { return own + (i / VECW) * kRowThreads * VECW + i % VECW; };
    float x[PER];
    if (base + kRowThreads * PER <= a.vocab) {
#pragma unroll
        for (int j = 0; j < PER / VECW; ++j) {
            const int64_t at = row_at + base + token_of(j * VECW);
            if constexpr (VECW == 1) x[j] = Elem<IO>::load(a.logits, at);
            else Vec<IO, VECW>::load(a.logits, at, &x[j * VECW]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < PER / VECW; ++j) {
            const int v = base + (int)token_of(j * VECW);
            if (VECW > 1 && v + VECW <= a.vocab) {
                if constexpr (VECW > 1) Vec<IO, VECW>::load(a.logits, row_at + v, &x[j * VECW]);
            } else {
#pragma unroll
                for (int e = 0; e < VECW; ++e)
                    x[j * VECW + e] = v + e < a.vocab ? Elem<IO>::load(a.logits, row_at + v + e) : kNone;
            }
        }
    }
    float gmax[G], top = kNone;  // fmaxf passes over NaN
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float* p = &x[g * 8];
        gmax[g] = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
        gmax[g] = fmaxf(gmax[g], kNone) + 0.0f;  // -0 counts as 0
        top = fmaxf(top, gmax[g]);
    }

    // sum of exponentials about the thread's own maximum, eight at a time in 32 bits
    const bool some = top > kNone;
    const float about = some ? top : 0.0f;
    double sum = sum_about<PER, false>(x, about);
    if (sum != sum) sum = sum_about<PER, true>(x, about);  // a NaN logit counts as -inf
    const float wtop = wave_max(top);
    sum = wave_sum(some ? sum * (double)exp_f32(top - wtop) : 0.0);

    sh_key[tid] = key_of(top);
    if (lane == 0) {
        sh_sum[tid >> 6] = sum;
        sh_top[tid >> 6] = wtop;
    }
    __syncthreads();
    // tau: a logit that at least `out` threads reach or pass, the out-th best of the threads' maxima.  (With the
    // best of the four waves' own such values a wave listed 13 logits instead of 4, and ranked 50 instead of 16.)
    uint32_t key[kRowWaves], tau_key = 0;
#pragma unroll
    for (int i = 0; i < kRowWaves; ++i) key[i] = sh_key[i * 64 + lane];
    constexpr int kLowBit = Elem<IO>::bytes == 2 ? 16 : 0;
#pragma unroll 4
    for (int bit = 31; bit >= kLowBit; --bit) {
        const uint32_t t = tau_key | (1u << bit);
        int c = 0;
#pragma unroll
        for (int i = 0; i < kRowWaves; ++i) c += __popcll(__ballot(key[i] >= t));
        if (c >= a.out) tau_key = t;
    }
    if (!(tau_key >> 31)) tau_key |= (1u << kLowBit) - 1;  // the keys of negative bf16 values end in ones
    if (tid == 0) {
        float btop = sh_top[0];
#pragma unroll
        for (int i = 1; i < kRowWaves; ++i) btop = fmaxf(btop, sh_top[i]);
        double s = 0.0;
        for (int i = 0; i < kRowWaves; ++i)
            if (sh_top[i] > kNone) s += sh_sum[i] * (double)exp_f32(sh_top[i] - btop);
        a.sums[(int64_t)row * a.splits + split] = s;
        a.tops[(int64_t)row * a.splits + split] = btop;
    }

    // Each wave lists its logits from tau on (-inf is never listed).  Where these are very many (few threads hold
    // them, or many are equal), tau becomes the wave's out-th best: those above it are listed again, and of those
    // equal to it the first `out` in the order of the tokens.
    float from = fmaxf(of_key(tau_key), -3.402823466e38f);
    uint64_t* mylist = list[tid >> 6];
    int found, ties = 0;
    for (bool exact = false;; exact = true) {
#pragma unroll
        for (int i = 0; i < PER; ++i) hide(x[i]);
        asm volatile("" : "+v"(own));  // nor are 64 token numbers kept from pass to pass
        found = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (!__ballot(gmax[g] >= from)) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool take = x[g * 8 + e] >= from;
                const uint64_t m = __ballot(take);
                if (!m) continue;
                const int at = found + lanes_below(m);
                if (take && at < kWaveCap) mylist[at] = entry_of(x[g * 8 + e] + 0.0f, base + token_of(g * 8 + e));
                found += __popcll(m);
            }
        }
        if (exact || found <= kWaveCap) break;
        uint32_t t = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const float u = of_key(t | (1u << bit));
            int c = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) c += __popcll(__ballot(x[i] >= u));
            if (c >= a.out) t |= 1u << bit;
        }
        const float tau = of_key(t);
        from = of_key(t + 1);  // the next float: fewer than `out` reach it
        int equal = 0;
#pragma unroll
        for (int j = 0; j < PER / VECW; ++j) {
            if (equal >= a.out || !__ballot(gmax[j * VECW / 8] >= tau)) continue;
            int n = 0;
#pragma unroll
            for (int e = 0; e < VECW; ++e) n += x[j * VECW + e] == tau;
            if (!__ballot(n > 0)) continue;
            // equal ones in lower lanes come first, then this lane's in order
            const int incl = (int)wave_inclusive_sum((float)n);
            int rank = equal + incl - n;
#pragma unroll
            for (int e = 0; e < VECW; ++e)
                if (x[j * VECW + e] == tau) {
                    if (rank < a.out) mylist[kBeamMaxOut + rank] = entry_of(tau + 0.0f, base + token_of(j * VECW + e));
                    ++rank;
                }
            equal += __builtin_amdgcn_readlane(incl, 63);
        }
        ties = min(equal, a.out);
    }
    if (ties > 0) {  // they stand behind room for `out` better ones
        uint64_t e = 0;
        if (lane < ties) e = mylist[kBeamMaxOut + lane];
        if (lane < ties) mylist[found + lane] = e;
        found += ties;
    }
    if (lane < 8) mylist[found + lane] = 0;  // to a multiple of eight: an entry better than none
    if (lane == 0) listed[tid >> 6] = found;
    __syncthreads();
    // an entry's place is the number of better ones
    uint64_t* out = a.entries + ((int64_t)row * a.splits + split) * a.out;
    int before[kRowWaves], all = 0;
#pragma unroll
    for (int v = 0; v < kRowWaves; ++v) {
        before[v] = all;
        all += listed[v];
    }
    if (all <= 64) {
        if (tid >= 64) return;
        uint64_t mine = 0;
#pragma unroll
        for (int v = 0; v < kRowWaves; ++v)
            if (lane >= before[v] && lane - before[v] < listed[v]) mine = list[v][lane - before[v]];
        int rank = 0;
        for (int j = 0; j < all; ++j) {
            const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)mine, j), hi = __builtin_amdgcn_readlane((uint32_t)(mine >> 32), j);
            rank += ((uint64_t)hi << 32 | lo) > mine;
        }
        if (lane < all && rank < a.out) out[rank] = mine;
        if (lane >= all && lane < a.out) out[lane] = 0;
        return;
    }
    for (int i = lane; i < found; i += 64) {
        const uint64_t mine = mylist[i];
        int rank = 0;
        for (int v = 0; v < kRowWaves; ++v) {
            const int n = listed[v];
            for (int j = 0; j < n; j += 8)
#pragma unroll
                for (int k = 0; k < 8; ++k) rank += list[v][j + k] > mine;
        }
        if (rank < a.out) out[rank] = mine;
    }
}

__device__ __forceinline__ uint64_t key_of64(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double of_key64(uint64_t k) {
    return __longlong_as_double((int64_t)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

// A scored candidate; those in one list are all different.  Better ones come first: the higher score, then the
// higher `tie`, which holds the lower beam, the higher logit and the lower token, from its top bits down.  Of two
// entries of one list the one that stands first there is therefore the better candidate, also where their scores
// round to the same value: how many candidates the merge can hold follows from it.
static_assert(kBeamMaxBeams <= 32 && kBeamMaxVocab <= 1 << 20, "5 bits of beam, 32 of logit, 20 of token");
constexpr uint32_t kTokenBits = (1u << 20) - 1;
struct __align__(16) Candidate {
    uint64_t key;
    uint64_t tie;
    __device__ __forceinline__ bool before(const Candidate& o) const {
        return key > o.key || (key == o.key && tie > o.tie);
    }
    __device__ __forceinline__ uint32_t beam() const { return kBeamMaxBeams - 1 - (uint32_t)(tie >> 52); }
    __device__ __forceinline__ uint32_t token() const { return ~(uint32_t)tie & kTokenBits; }
};
__device__ __forceinline__ uint64_t tie_of(int w, uint32_t logit_key, uint32_t token) {
    return (uint64_t)(kBeamMaxBeams - 1 - w) << 52 | (uint64_t)logit_key << 20 | (~token & kTokenBits);
}

// Sorts the first n of an LDS list, n <= kMergeThreads by counting, more by a network over the next power of
// two.  Counting: kMergeThreads / n threads per candidate share the comparisons, and each reads eight ahead of
// comparing them (one at a time it waited for the LDS in every step: 32 candidates took 8000 cycles).  `rank`
// is LDS scratch of kMergeThreads.
__device__ __forceinline__ void sort_candidates(Candidate* list, int n, int* rank) {
    if (n <= kMergeThreads) {
        const int tid = threadIdx.x, np = pow2_at_least(n), parts = kMergeThreads / np;
        const int i = tid & (np - 1), part = tid / np, each = (n + parts - 1) / parts;
        const int j0 = part * each, j1 = min(n, j0 + each);
        Candidate mine{0, 0};
        if (i < n) mine = list[i];
        rank[tid] = 0;
        int before = 0;
#pragma unroll 8
        for (int j = j0; j < j1; ++j) before += list[j].before(mine);
        __syncthreads();
        if (i < n && before) atomicAdd(&rank[i], before);
        __syncthreads();
        if (tid < n) list[rank[tid]] = mine;  // part 0: candidate tid
        __syncthreads();
        return;
    }
    const int np = pow2_at_least(n);
    for (int i = n + threadIdx.x; i < np; i += kMergeThreads) list[i] = Candidate{0, 0};
    bitonic_sort<kMergeThreads>(np, [&](int i, int j, bool down) {
        const Candidate p = list[i], q = list[j];
        if (q.before(p) == down) {
            list[i] = q;
            list[j] = p;
        }
    });
}

// Bound by its chain of dependent steps, not by data: one search of 4 beams over 32000 4.8 us, 32 of 8 over 131072
// 8.0 us.
template <typename IO> __global__ __launch_bounds__(kMergeThreads) void beam_merge_kernel(const BeamArgs a) {
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    constexpr int kWavesM = kMergeThreads / 64, kHeld = 8 * kMergeThreads;
    const int W = a.beams, S = a.splits, K = a.out, lists = W * S, total = lists * K;
    const float kNone = -__builtin_inff();
    extern __shared__ __align__(16) char smem[];
    Candidate* best = reinterpret_cast<Candidate*>(smem);                     // [merge_list]
    __shared__ double lse[kBeamMaxBeams], red[kWavesM];
    __shared__ float beam_score[kBeamMaxBeams];
    __shared__ int state[kBeamMaxBeams];                                      // 0: listed, 1: ended, 2: no candidates
    static_assert(kBeamMaxBeams <= 64, "a lane per beam");
    __shared__ int rank[kMergeThreads];
    __shared__ int count;
    __shared__ uint32_t near_mask, behind_mask, tau_mask;                     // a bit per beam

    // the first entries go to the LDS, in flight with the sums
    const uint64_t* entries = a.entries + (int64_t)b * total;
    __shared__ uint64_t held[kHeld];
    uint64_t mine[kHeld / kMergeThreads];
#pragma unroll
    for (int r = 0; r < kHeld / kMergeThreads; ++r) {
        const int i = tid + r * kMergeThreads;
        mine[r] = i < total ? entries[i] : 0;
    }
    // log-sum-exp per beam: a row of 16 lanes holds its parts, or a wave
    const int width = S <= 16 ? 16 : 64, per_wave = 64 / width;
    for (int w0 = wave * per_wave; w0 < W; w0 += kWavesM * per_wave) {
        const int w = w0 + lane / width, part = lane & (width - 1);
        const bool in = w < W;
        const int64_t row = (int64_t)b * W + (in ? w : 0);
        const float score = a.scores[row];
        const bool ended = a.finished && a.finished[row];
        const float m = in && part < S ? a.tops[row * S + part] : kNone;
        const double mass = in && part < S ? a.sums[row * S + part] : 0.0;
        const float top = width == 16 ? row16_max(m) : wave_max(m);
        // a part without a finite logit has the sum of nothing; rows of ended beams hold no parts
        double sum = m > kNone ? mass * (double)exp_f32(m - top) : 0.0;
        sum = width == 16 ? row16_sum64(sum) : wave_sum(sum);
        if (in && part == 0) {
            const bool real = score > kNone && score < -kNone, finite = top > kNone && top < -kNone;
            state[w] = !real ? 2 : ended ? 1 : finite ? 0 : 2;
            lse[w] = (double)top + log(sum);
            beam_score[w] = score;
        }
    }
#pragma unroll
    for (int r = 0; r < kHeld / kMergeThreads; ++r) held[tid + r * kMergeThreads] = mine[r];
    __syncthreads();

    // entry i's candidate; false: none
    const float per_beam = 1.0f / (float)(S * K);
    auto candidate = [&](int i, uint64_t e, Candidate& c) {
        const int w = (int)(((float)i + 0.5f) * per_beam);  // i / (S K): exact for i < 2^21
        const double score = (double)beam_score[w];
        if (state[w] == 1 && i == w * S * K) {
            c = Candidate{key_of64(score), tie_of(w, 0, a.eos)};
            return true;
        }
        if (state[w] != 0 || !e) return false;
        const uint32_t logit = (uint32_t)(e >> 32);
        c = Candidate{key_of64(score + ((double)of_key(logit) - lse[w])), tie_of(w, logit, ~(uint32_t)e)};
        return true;
    };
    auto entry = [&](int i) { return i < kHeld ? held[i] : entries[i]; };
    int n = 0;
    for (int pass = 0; pass < 2; ++pass) {
        Candidate tau{0, 0};
        // with more lists than results, no result and not the one behind them comes after the (K+1)-th best of
        // the lists' first entries, and at most K lists hold better ones
        if (lists > K) {
            for (int l = tid; l < lists; l += kMergeThreads) {
                Candidate c{0, (uint64_t)l};  // an empty list stands behind all others, at a place of its own
                candidate(l * K, entry(l * K), c);
                best[l] = c;
            }
            __syncthreads();
            sort_candidates(best, lists, rank);
            tau = best[K];
        }
        if (tid == 0) {
            count = 0;
            near_mask = behind_mask = tau_mask = 0;
        }
        __syncthreads();
        for (int i = tid; i < total; i += kMergeThreads) {
            Candidate c;
            if (!candidate(i, entry(i), c)) continue;
            if (c.before(tau)) {
                const int at = atomicAdd(&count, 1);
                if (at < a.merge_list) best[at] = c;  // more are only there if another call writes this workspace
            } else if (near_scores(of_key64(tau.key), of_key64(c.key))) {
                atomicOr(&tau_mask, 1u << c.beam());
            }
        }
        __syncthreads();
        n = min(count, a.merge_list);
        if (tau.key && n <= K) {
            if (tid == 0) best[n] = tau;
            ++n;
            __syncthreads();
        }
        sort_candidates(best, n, rank);
        if (pass == 1) break;
        // neighbours of the result, and what is near its last one: one beam's equal logits may stand between that
        // and another beam's, in the list or not listed because they stand behind tau
        const double last = n >= K ? of_key64(best[K - 1].key) : 0.0;
        for (int i = tid; i < n; i += kMergeThreads) {
            const uint32_t w0 = best[i].beam();
            if (i + 1 < min(n, K)) {
                const uint32_t w1 = best[i + 1].beam();
                if (w0 != w1 && near_scores(of_key64(best[i].key), of_key64(best[i + 1].key)))
                    atomicOr(&near_mask, (1u << w0) | (1u << w1));
            } else if (i >= K - 1 && near_scores(last, of_key64(best[i].key))) {
                atomicOr(&behind_mask, 1u << w0);
            }
        }
        __syncthreads();
        uint32_t behind = behind_mask, near = near_mask;
        if (n >= K && near_scores(last, of_key64(tau.key))) behind |= tau_mask;
        if (behind & (behind - 1)) near |= behind;  // more than one beam
        near &= (uint32_t)__ballot(lane < W && state[lane < W ? lane : 0] == 0);  // an ended beam's score has no sum
        near = __builtin_amdgcn_readfirstlane(near);  // one value: the loop over beams stays scalar (401 us, 408 without)
        __syncthreads();  // every wave has read the masks before they are cleared, and all go on or none
        if (!near) break;
        for (int w = 0; w < W; ++w) {
            if (!((near >> w) & 1)) continue;
            const int64_t at = ((int64_t)b * W + w) * a.stride;
            float top = kNone;
            for (int s = 0; s < S; ++s) top = fmaxf(top, a.tops[((int64_t)b * W + w) * S + s]);
            double sum = 0.0;
            // eight logits in flight per thread: 50 us a beam of 131072 (185 one at a time)
#pragma unroll 8
            for (int v = tid; v < a.vocab; v += kMergeThreads)
                sum += exp((double)clean(Elem<IO>::load(a.logits, at + v)) - (double)top);
            sum = wave_sum(sum);
            if (lane == 0) red[wave] = sum;
            __syncthreads();
            if (tid == 0) {
                double s = 0.0;
                for (int i = 0; i < kWavesM; ++i) s += red[i];
                lse[w] = (double)top + log(s);
            }
            __syncthreads();
        }
    }
    const int have = min(n, K);
    for (int i = tid; i < have; i += kMergeThreads) {
        a.out_scores[(int64_t)b * K + i] = (float)of_key64(best[i].key);
        a.out_parents[(int64_t)b * K + i] = best[i].beam();
        a.out_tokens[(int64_t)b * K + i] = best[i].token();
    }
    // fewer candidates than asked for: those of probability zero follow, by the lower index
    if (have == K || wave != 0) return;
    int at = have;
    for (int w = 0; w < W && at < K; ++w) {
        const int64_t row = ((int64_t)b * W + w) * a.stride;
        for (int v0 = 0; v0 < a.vocab && at < K; v0 += 64) {
            const int v = v0 + lane;
            bool none = v < a.vocab;
            if (none && state[w] == 1) none = v != a.eos;
            if (none && state[w] == 0) none = clean(Elem<IO>::load(a.logits, row + v)) == -__builtin_inff();
            const uint64_t m = __ballot(none);
            const int p = at + lanes_below(m);
            if (none && p < K) {
                a.out_scores[(int64_t)b * K + p] = -__builtin_inff();
                a.out_parents[(int64_t)b * K + p] = w;
                a.out_tokens[(int64_t)b * K + p] = v;
            }
            at += __popcll(m);
        }
    }
}

// ---- reordering ----
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

// HBM-bound.  94 copies of 2 MiB states: 63 us with 16 KiB per workgroup and non-temporal stores; 72 with ordinary
// stores, 69 with non-temporal loads too, 115 to 137 with 32 KiB per workgroup, whatever the loads and stores.  201 MB
// are written and 143 read (a parent's copies share one read through the caches): 5.4 TB/s.
// One workgroup per (part of a slot, child, layer); every wave works out the child's slot for itself.
template <typename T> __global__ __launch_bounds__(kCopyThreads) void beam_reorder_kernel(const ReorderArgs a) {
    const int child = blockIdx.y % a.beams, b = blockIdx.y / a.beams;
    const int lane = threadIdx.x & 63;
    const bool in = lane < a.beams;
    const int parent = in ? a.parents[b * a.beams + lane] : -1;
    const int slot = in ? a.slots[b * a.beams + lane] : -1;
    const bool wrong = in && ((unsigned)parent >= (unsigned)a.beams || (unsigned)slot >= (unsigned)a.num_slots);
    const int my_parent = __builtin_amdgcn_readlane(parent, child);
    const bool head = blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0;
    if (__ballot(wrong)) {  // a padded row: its slots stay
        if (head) a.slots_out[b * a.beams + child] = __builtin_amdgcn_readlane(slot, child);
        return;
    }
    uint64_t childless = 0, first = 0;
    for (int p = 0; p < a.beams; ++p) {
        const uint64_t m = __ballot(parent == p);
        if (m) first |= m & -m; else childless |= 1ull << p;
    }
    const int src = __builtin_amdgcn_readlane(slot, my_parent);
    int dst = src;
    if (!((first >> child) & 1)) {
        int rank = __popcll(~first & ((1ull << child) - 1));
        while (rank-- > 0) childless &= childless - 1;
        dst = __builtin_amdgcn_readlane(slot, __builtin_ctzll(childless));
    }
    if (head) a.slots_out[b * a.beams + child] = dst;
    if (dst == src) return;
    const int64_t units = a.slot_bytes / sizeof(T);
    char* layer = a.pool + (int64_t)blockIdx.z * a.layer_bytes;
    const T* from = reinterpret_cast<const T*>(layer + (int64_t)src * a.slot_bytes);
    T* to = reinterpret_cast<T*>(layer + (int64_t)dst * a.slot_bytes);
    const int64_t i0 = (int64_t)blockIdx.x * (kCopyThreads * kCopyUnroll) + threadIdx.x;
    T r[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
        if (i0 + u * kCopyThreads < units) r[u] = from[i0 + u * kCopyThreads];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
        if (i0 + u * kCopyThreads < units) __builtin_nontemporal_store(r[u], to + i0 + u * kCopyThreads);
}

template <typename T> hipError_t reorder(const ReorderArgs& a, hipStream_t s) {
    const int64_t units = a.slot_bytes / sizeof(T), per = kCopyThreads * kCopyUnroll;
    const int64_t parts = (units + per - 1) / per;
    if (parts >= (1ll << 32) / kCopyThreads) return hipErrorInvalidValue;  // a launch has fewer than 2^32 threads
    beam_reorder_kernel<T><<<dim3((unsigned)parts, (unsigned)(a.batch * a.beams), (unsigned)a.layers), kCopyThreads, 0, s>>>(a);
    return hipGetLastError();
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

template <typename IO, int PER> hipError_t rows(const BeamArgs& a, hipStream_t s) {
    constexpr int VECW = 16 / Elem<IO>::bytes;
    const dim3 grid(a.splits, a.batch * a.beams);
    if (a.stride % VECW == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0)
        beam_rows_kernel<IO, PER, VECW><<<grid, kRowThreads, 0, s>>>(a);
    else
        beam_rows_kernel<IO, PER, 1><<<grid, kRowThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <typename IO> hipError_t select(BeamArgs a, const BeamPlan& pl, hipStream_t s) {
    hipError_t e = pl.per_thread == 16 ? rows<IO, 16>(a, s) : pl.per_thread == 32 ? rows<IO, 32>(a, s) : rows<IO, 64>(a, s);
    if (e != hipSuccess) return e;
    // the merge keeps the entries of at most `out` lists, `out` each, and one more where these are fewer than
    // out + 1; the lists' first entries stand there before
    int most = a.out * a.out;
    const int lists = a.beams * a.splits;
    if (most < lists) most = lists;
    if (most < a.out + 1) most = a.out + 1;
    a.merge_list = 2;
    while (a.merge_list < most) a.merge_list *= 2;
    beam_merge_kernel<IO><<<a.batch, kMergeThreads, (size_t)a.merge_list * sizeof(Candidate), s>>>(a);
    return hipGetLastError();
}

}  // namespace

// Parts of 4096, 8192 or 16384 logits: the largest that still gives the part two workgroups per CU, and
// at most kMaxSplits of them per row.
BeamPlan beam_plan(int32_t batch, int32_t beams, int32_t vocab, int32_t out) {
    BeamPlan pl{};
    const int64_t rows = (int64_t)batch * beams;
    pl.per_thread = 64;
    auto splits = [&](int per) { return (vocab + per * kRowThreads - 1) / (per * kRowThreads); };
    while (pl.per_thread > 16 && rows * splits(pl.per_thread) < 512 && splits(pl.per_thread / 2) <= kMaxSplits) pl.per_thread /= 2;
    pl.splits = splits(pl.per_thread);
    pl.chunk = pl.per_thread * kRowThreads;
    pl.sums = 0;
    pl.tops = up256((size_t)rows * pl.splits * sizeof(double));
    pl.entries = pl.tops + up256((size_t)rows * pl.splits * sizeof(float));
    pl.total = pl.entries + up256((size_t)rows * pl.splits * out * sizeof(uint64_t));
    return pl;
}

hipError_t launch_beam_select(const BeamArgs& args, const BeamPlan& pl, char* ws, int io_dtype, hipStream_t stream) {
    BeamArgs a = args;
    a.splits = pl.splits;
    a.chunk = pl.chunk;
    a.sums = reinterpret_cast<double*>(ws + pl.sums);
    a.tops = reinterpret_cast<float*>(ws + pl.tops);
    a.entries = reinterpret_cast<uint64_t*>(ws + pl.entries);
    return io_dtype == 0 ? select<float>(a, pl, stream) : select<bf16_t>(a, pl, stream);
}

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t s) {
    const uintptr_t both = reinterpret_cast<uintptr_t>(a.pool) | (uintptr_t)a.slot_bytes;
    if (both % 16 == 0) return reorder<u32x4_t>(a, s);
    if (both % 4 == 0) return reorder<uint32_t>(a, s);
    return reorder<uint16_t>(a, s);
}

}  // namespace gdr
