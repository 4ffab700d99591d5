// Gated linear recurrence (one state value per channel) for gfx950: scan over a packed varlen batch,
// its backward pass, and the paged decode form.
//
//   h_t = a_t h_{t-1} + b_t,  y_t = h_t     log gate: a = e^g, b = x;  sigmoid gate: a = s(z), b = (1 - a) x
//   D_t = dy_t + a_{t+1} D_{t+1}            (+ the final state's gradient at a sequence's last token)
//   log: dx = D, dg = D a h_{t-1};  sigmoid: dx = (1 - a) D, dz = D a (1 - a) (h_{t-1} - x);  dh0 = a_1 D_1
//
// A run of tokens maps the state before it to the state behind it as h -> A h + B, and runs compose:
// (A2, B2) after (A1, B1) is (A2 A1, A2 B1 + B2).  A sequence's first token replaces the carried state
// by the initial state, so a run that holds one no longer depends on what came before: it is marked as
// cut, and everything that applies a run tests the mark instead of multiplying by 0, so that an infinity
// or a NaN of one sequence never reaches the next.  The packed token axis is cut into tiles whatever the
// sequences' borders are.  The backward pass composes the same way from the right (c_t = a_t (dy_t +
// c_{t+1}), cut at each sequence's last token).
//
// Layout: a lane owns VEC neighbouring channels, a wave a run of TPT tokens, the W waves of a workgroup
// the W runs of a tile; a lane holds its channels' rows in registers and walks them in time order, so no
// value crosses lanes and every input is read once.  A large batch is bound by HBM and by how well the loads of
// one workgroup cover the arithmetic of the other on its CU (32768 x 4096 bf16, log gate: 207 us, 5.2 TB/s, VALU
// busy half the time; 65573 x 2048 fp32, one sequence: 284 us, 5.7 TB/s), a small one by the latency of a tile.
#include "gdr_device.h"
#include "gdr_internal.h"

namespace gdr {

namespace {

constexpr int kWavesPerSimd = 4;        // two workgroups of 8 waves per CU: at most 128 registers
constexpr int kLogGate = 0;

// ---- a lane's VEC channels of one token, as loaded ----
template <typename T, int VEC> struct Chan;
template <> struct Chan<float, 4> {
    f32x4_t v;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        v = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kNonTemporal));
    }
    __device__ __forceinline__ void get(float* out) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = v[e];
    }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(v)); }
    __device__ __forceinline__ static void put(__amdgpu_buffer_rsrc_t r, uint32_t off, const float* in) {
        BufStore<float, 4>::store<kNonTemporal>(r, off, in);
    }
};
template <> struct Chan<bf16_t, 4> {
    u32x2_t w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        w = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, kNonTemporal));
    }
    __device__ __forceinline__ void get(float* out) const {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            out[2 * e] = __uint_as_float(w[e] << 16);
            out[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(w)); }
    __device__ __forceinline__ static void put(__amdgpu_buffer_rsrc_t r, uint32_t off, const float* in) {
        BufStore<bf16_t, 4>::store<kNonTemporal>(r, off, in);
    }
};
template <> struct Chan<float, 2> {
    u32x2_t w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        w = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, kNonTemporal));
    }
    __device__ __forceinline__ void get(float* out) const {
        out[0] = __uint_as_float(w[0]);
        out[1] = __uint_as_float(w[1]);
    }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(w)); }
    __device__ __forceinline__ static void put(__amdgpu_buffer_rsrc_t r, uint32_t off, const float* in) {
        __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{__float_as_uint(in[0]), __float_as_uint(in[1])}, r, off, 0, kNonTemporal);
    }
};
template <> struct Chan<bf16_t, 2> {
    uint32_t w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        w = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, kNonTemporal);
    }
    __device__ __forceinline__ void get(float* out) const {
        out[0] = __uint_as_float(w << 16);
        out[1] = __uint_as_float(w & 0xFFFF0000u);
    }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(w)); }
    __device__ __forceinline__ static void put(__amdgpu_buffer_rsrc_t r, uint32_t off, const float* in) {
        __builtin_amdgcn_raw_buffer_store_b32(pack_bf16x2(in[0], in[1]), r, off, 0, kNonTemporal);
    }
};
template <> struct Chan<float, 1> {
    uint32_t w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        w = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, kNonTemporal);
    }
    __device__ __forceinline__ void get(float* out) const { out[0] = __uint_as_float(w); }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(w)); }
    __device__ __forceinline__ static void put(__amdgpu_buffer_rsrc_t r, uint32_t off, const float* in) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(in[0]), r, off, 0, kNonTemporal);
    }
};
template <> struct Chan<bf16_t, 1> {
    uint32_t w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
        w = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, kNonTemporal);
    }
    __device__ __forceinline__ void get(float* out) const { out[0] = __uint_as_float(w << 16); }
    __device__ __forceinline__ void hide() { asm volatile("" : "+v"(w)); }
    __device__ __forceinline__ static void put(__amdgpu_buffer_rsrc_t r, uint32_t off, const float* in) {
        __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(in[0]), r, off, 0, kNonTemporal);
    }
};

// A wave's rows of a [T, D] tensor: token w0 + i, this lane's channels.  The resource ends behind the last
// valid row, and lanes without channels get an offset behind every resource, so that reads there give zeros
// and writes nothing without a branch (32 rows of at most 2^22 channels keep every offset below 2^30).
template <typename T> struct Rows {
    __amdgpu_buffer_rsrc_t r;
    uint32_t off, row;
    __device__ __forceinline__ Rows(const void* p, int64_t D, int64_t w0, int rows, int64_t c, bool active) {
        constexpr int B = Elem<T>::bytes;
        char* base = const_cast<char*>(static_cast<const char*>(p)) + w0 * D * B;
        r = __builtin_amdgcn_make_buffer_rsrc(base, 0, (int)(rows * D * B), 0x00020000);
        off = active ? (uint32_t)(c * B) : 0x80000000u;
        asm volatile("" : "+v"(off));  // another tensor's offsets are not kept for this one's
        row = (uint32_t)(D * B);
    }
    __device__ __forceinline__ uint32_t at(int i) const { return off + i * row; }
};

template <int KIND, typename IO> struct GateT { typedef IO T; };
template <typename IO> struct GateT<kLogGate, IO> { typedef float T; };

// ---- decays ----
// A channel that forgets 1e-4 of its state per token needs that 1e-4 to more than the 2^-24 of 1 that a
// rounded a holds: the error repeats every token and would grow to 2^-24 / 1e-4 of the result.  A decay is
// therefore held as one float whose sign says which form it is: v = 1 - a >= +0 where a is near 1, v = -a
// elsewhere.  Either way a h = (v's sign clear ? h : 0) - v h, one select and one fma.  (An infinite state
// becomes a NaN at its next step: a h is inf - inf.)
__device__ __forceinline__ bool near_one(float v) { return (int)__float_as_uint(v) >= 0; }
__device__ __forceinline__ float mul_a(float v, float h) { return fmaf(-v, h, near_one(v) ? h : 0.0f); }
__device__ __forceinline__ float one_minus(float v) { return near_one(v) ? v : 1.0f + v; }

__device__ __forceinline__ float encode_log(float g) {
    // -1/16 < g <= -0: 1 - e^g by its series (the next term is 1e-9 of the result); +0 gives a = 1.  Beyond,
    // the rounding of a is at most 2^-23 / 0.06 = 2e-6 of the decay.
    float p = fmaf(g, 1.0f / 120.0f, 1.0f / 24.0f);
    p = fmaf(g, p, 1.0f / 6.0f);
    p = fmaf(g, p, 0.5f);
    p = fmaf(g, p, 1.0f);
    const bool near = __float_as_uint(g) - 0x80000000u < 0x3D800000u;
    return near ? fabsf(g * p) : -exp_f32(g);
}

__device__ __forceinline__ float encode_sigmoid(float z) {
    const float e = exp_f32(-fabsf(z));
    return __builtin_copysignf(e * __builtin_amdgcn_rcpf(1.0f + e), z);  // the smaller of a and 1 - a
}

template <int KIND> __device__ __forceinline__ float encode_gate(float raw) {
    return KIND == kLogGate ? encode_log(raw) : encode_sigmoid(raw);
}

// h_t from h_{t-1}: a h + x, or a h + (1 - a) x = (near 1 ? h : x) - v (h - x)
template <int KIND> __device__ __forceinline__ float step(float v, float h, float x) {
    if constexpr (KIND == kLogGate) return mul_a(v, h) + x;
    return fmaf(-v, h - x, near_one(v) ? h : x);
}

// ---- runs: (v, B), v the whole run's decay in the same form, or kCut ----
constexpr float kCut = __builtin_inff();

// The state behind a run entered with state h.
__device__ __forceinline__ float apply_run(float2 r, float h) { return r.x == kCut ? r.y : mul_a(r.x, h) + r.y; }

// 1 - A is kept where it is small and A where that is: a product of rounded decays near 1 would lose
// their complements as a single rounded decay does.
__device__ __forceinline__ float pick(float A, float Q) { return Q >= 0.0f && Q < 0.125f ? fabsf(Q) : -A; }

__device__ __forceinline__ float2 compose(float2 r1, float2 r2) {
    if (r2.x == kCut) return r2;
    const float B = mul_a(r2.x, r1.y) + r2.y;
    if (r1.x == kCut) return float2{kCut, B};
    const float q1 = one_minus(r1.x), a1 = near_one(r1.x) ? 1.0f - r1.x : -r1.x;
    return float2{pick(mul_a(r2.x, a1), fmaf(one_minus(r2.x), 1.0f - q1, q1)), B};
}

// The decay of a run of gates: the log gates' sum, or the product of the decays beside its complement.
// Each is summed as the run is walked, not from 64 kept gates at the end.
template <int KIND> struct RunDecay;
template <> struct RunDecay<kLogGate> {
    float G = 0.0f;
    __device__ __forceinline__ void add(float raw, float) {
        G += raw;
        hide(G);
    }
    __device__ __forceinline__ float get() const { return encode_log(G); }
};
template <> struct RunDecay<1> {
    float A = 1.0f, Q = 0.0f;
    __device__ __forceinline__ void add(float, float v) {
        A = mul_a(v, A);
        Q = fmaf(v, 1.0f - Q, near_one(v) ? Q : 1.0f);
        hide(A);
        hide(Q);
    }
    __device__ __forceinline__ float get() const { return pick(A, Q); }
};

// ---- which of a wave's TPT tokens begin and end a sequence ----
struct Borders {
    uint64_t first, last;  // bit i: token w0 + i is the first / last of its sequence
    int n;                 // lane i: the sequence of token w0 + i
    __device__ __forceinline__ int seq(int i) const { return __builtin_amdgcn_readlane(n, i); }
};

// cu_seqlens is read with scalar loads: their results do not queue behind the tile's vector loads.
typedef const __attribute__((address_space(4))) int32_t* ScalarInts;
__device__ __forceinline__ ScalarInts scalar_ints(const int32_t* p) { return (ScalarInts)(uintptr_t)p; }

__device__ __forceinline__ int64_t tokens_end(const LinearArgs& a) {
    if (!a.cu) return a.T;
    const int64_t e = scalar_ints(a.cu)[a.N];
    return e < a.T ? e : a.T;
}

template <int TPT> __device__ __forceinline__ Borders find_borders(const LinearArgs& a, int64_t w0, int64_t end) {
    static_assert(TPT <= 64, "one lane per token");
    Borders b{0, 0, 0};
    const int lane = threadIdx.x & 63;
    if (!a.cu) {
        if (w0 == 0) b.first = 1;
        if (w0 < end && end <= w0 + TPT) b.last = 1ull << (end - 1 - w0);
        return b;
    }
    if (w0 >= end) return b;
    const ScalarInts cu = scalar_ints(a.cu);
    int n = 0, hi = a.N;  // the last n < N with cu[n] <= w0: empty sequences at w0 come before it
    while (hi - n > 1) {
        const int mid = (n + hi) >> 1;
        if (cu[mid] <= w0) n = mid; else hi = mid;
    }
    b.n = n;
    if (cu[n] == w0) b.first = 1;
    while (n < a.N) {  // sequences that end in this run of tokens
        const int64_t e = cu[n + 1];
        if (e > w0 + TPT || e > end) break;
        if (e > w0 && e > cu[n]) b.last |= 1ull << (e - 1 - w0);
        if (++n == a.N || e == w0 + TPT || e == end) break;
        if (e > w0 && cu[n + 1] > e) b.first |= 1ull << (e - w0);
        if (lane >= e - w0) b.n = n;
    }
    return b;
}

template <int TPT> __device__ __forceinline__ int rows_of(int64_t w0, int64_t end) {
    return end <= w0 ? 0 : end - w0 < TPT ? (int)(end - w0) : TPT;
}

// Row n of a [N, D] fp32 tensor, this lane's channels; without a tensor, and for lanes without channels, zeros.
template <int VEC> __device__ __forceinline__ void load_state(const float* p, int64_t n, int64_t D, int64_t c, float* out) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = 0.0f;
    if (p && c < D) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = p[n * D + c + e];
    }
}
template <int VEC> __device__ __forceinline__ void store_state(float* p, int64_t n, int64_t D, int64_t c, const float* in) {
    if (p && c < D) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[n * D + c + e] = in[e];
    }
}

// Empty sequences have no token whose lane could write their final state (or its gradient): the workgroup
// of the chain's first tile copies them, VEC channels per lane, a sequence per wave.
template <int VEC, int W> __device__ __forceinline__ void copy_empty(const LinearArgs& a, const float* src, float* dst, int64_t c) {
    if (!a.cu || !dst) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int n0 = w * 64; n0 < a.N; n0 += W * 64) {
        const int n = n0 + lane;
        uint64_t m = __ballot(n < a.N && a.cu[n < a.N ? n : 0] == a.cu[n < a.N ? n + 1 : 0]);
        for (; m; m &= m - 1) {
            const int s = n0 + __builtin_ctzll(m);
            float h[VEC];
            load_state<VEC>(src, s, a.D, c, h);
            store_state<VEC>(dst, s, a.D, c, h);
        }
    }
}

// ---- the states between tiles ----
// A tile publishes its run as soon as it has it, looks at the runs of the 8 tiles before it until one of them
// is cut, and publishes the state behind itself as a cut run.  A word is one 64-bit value, written and
// read whole at device scope, so it needs no flag and no fence: its decay is kEmpty until it is written.
// Tiles are handed out by a counter in the order of the chain, so a tile waits only for tiles whose workgroups
// have started.  These publish their runs without waiting for anything, the first one's is cut, and a tile
// whose predecessor's is cut publishes a cut one: every wait ends.
constexpr uint32_t kEmpty = 0xFFFFFFFFu;

__device__ __forceinline__ uint64_t* run_word(const LinearArgs& a, int64_t at, int64_t c) { return a.runs + at * a.D + c; }

__device__ __forceinline__ void publish(uint64_t* word, float2 r) {
    const uint32_t v = r.x == r.x ? __float_as_uint(r.x) : 0x7FC00000u;  // no NaN may read as kEmpty
    __hip_atomic_store(word, ((uint64_t)v << 32) | __float_as_uint(r.y), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ __launch_bounds__(256) void linear_init_kernel(const LinearArgs a, int64_t pairs) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i == 0) *a.ticket = 0;
    if (i < pairs) reinterpret_cast<uint4*>(a.runs)[i] = uint4{~0u, ~0u, ~0u, ~0u};
}

constexpr int kBack = 8;              // tiles that a tile looks back to

template <int VEC, int W> struct TileShared {
    float2 run[W][64 * VEC];         // the waves' runs; then the run of all waves before each
    float2 back[kBack][64 * VEC];    // runs of earlier tiles
    float carry[64 * VEC];           // the state entering the tile
    int ticket;
};

// Which tile of the chain this workgroup takes.
template <int VEC, int W> __device__ __forceinline__ int64_t take_ticket(const LinearArgs& a, TileShared<VEC, W>& sh) {
    if (a.tiles == 1) return blockIdx.x;
    if (threadIdx.x == 0) sh.ticket = (int)atomicAdd(a.ticket, 1u);
    __syncthreads();
    return sh.ticket;
}

// After every wave has stored its run (and a barrier): fills sh.carry and turns sh.run into the runs of all
// waves that come before each.  `at` is the tile's place in the chain; REVERSE: the waves' order is W-1 .. 0.
template <int VEC, int W, bool REVERSE>
__device__ __forceinline__ void chain(const LinearArgs& a, TileShared<VEC, W>& sh, int64_t at, int64_t c_tile) {
    static_assert(64 * W >= 64 * VEC && kBack % (W < kBack ? W : kBack) == 0, "a thread per channel, whole rounds of waves");
    constexpr int CH = 64 * VEC;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    float2 whole{0.0f, 0.0f};
    if (tid < CH) {
        float2 r = sh.run[REVERSE ? W - 1 : 0][tid];
#pragma unroll
        for (int i = 1; i < W; ++i) {
            float2& slot = sh.run[REVERSE ? W - 1 - i : i][tid];
            const float2 mine = slot;
            slot = r;
            r = compose(r, mine);
        }
        whole = r;
        if (at == 0) whole = float2{kCut, r.y};  // nothing comes before: entered with 0
        if (a.tiles > 1 && at + 1 < a.tiles && c_tile + tid < a.D) publish(run_word(a, at, c_tile + tid), whole);
        sh.carry[tid] = 0.0f;
    }
    if (at > 0) {
        // Wave w reads the word of the tile w + 1 places back.  The state is carried forward tile by tile; a cut run
        // sets it whatever stood before, so the nearest one decides.  That run's B is apply_run(whole, state) of the
        // same chain, so the state is the same, bit for bit, whichever of the tiles are cut already.  A pass
        // in which a channel meets no cut run gives it no state, and its words are looked at again.
        float state;
        for (;;) {
            state = 0.0f;
#pragma unroll
            for (int k = 0; k < kBack; k += W) {
                if (w + k >= kBack) break;
                const int64_t from = at - 1 - w - k;
                float2 got[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) got[e] = float2{kCut, 0.0f};
                if (from >= 0 && c_tile + lane * VEC < a.D) {
                    uint64_t word[VEC];
                    for (;;) {
                        bool empty = false;
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            word[e] = __hip_atomic_load(run_word(a, from, c_tile + lane * VEC + e), __ATOMIC_RELAXED,
                                                        __HIP_MEMORY_SCOPE_AGENT);
                            empty |= (uint32_t)(word[e] >> 32) == kEmpty;
                        }
                        if (!empty) break;
                        __builtin_amdgcn_s_sleep(1);
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        got[e] = float2{__uint_as_float((uint32_t)(word[e] >> 32)), __uint_as_float((uint32_t)word[e])};
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) sh.back[w + k][lane * VEC + e] = got[e];
            }
            __syncthreads();
            bool found = false;
            if (tid < CH) {
#pragma unroll
                for (int i = kBack - 1; i >= 0; --i) {
                    const float2 r = sh.back[i][tid];
                    found |= r.x == kCut;
                    state = apply_run(r, state);
                }
            }
            if (!__syncthreads_or(tid < CH && !found)) break;
        }
        if (tid < CH) {
            sh.carry[tid] = state;
            if (at + 1 < a.tiles && whole.x != kCut && c_tile + tid < a.D)
                publish(run_word(a, at, c_tile + tid), float2{kCut, apply_run(whole, state)});
        }
    }
    __syncthreads();
}

// =====================================================================================================
// forward.  Reads x and the gate, writes y, once each: 32768 x 4096 bf16 log 204 us (831 MB read, 277 written, VALU
// busy 47%), 65573 x 2048 fp32 280 us (33%), 16384 x 4096 bf16 sigmoid 101 us (4.2 TB/s, 50%).
template <int KIND, typename IO, int VEC, int W, int TPT>
__global__ __launch_bounds__(64 * W, kWavesPerSimd) void linear_fwd_kernel(const LinearArgs a) {
    constexpr int L = W * TPT;
    static_assert(L % kLinearBlock == 0, "the workspace holds a word per channel and block, block states begin runs");
    __shared__ TileShared<VEC, W> sh;
    const int64_t ticket = take_ticket(a, sh);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tile = ticket / a.nch;
    const int64_t c_tile = (ticket % a.nch) * (64 * VEC);
    const int64_t c = c_tile + lane * VEC;
    const bool active = c < a.D;  // with VEC > 1 a lane's channels exist all or none
    const int64_t end = tokens_end(a);
    const int64_t w0 = tile * L + (int64_t)w * TPT;

    typedef typename GateT<KIND, IO>::T GT;
    const int rows = rows_of<TPT>(w0, end);
    Chan<IO, VEC> x[TPT];
    float v[TPT][VEC];
    {
        const Rows<IO> rx(a.x, a.D, w0, rows, c, active);
        const Rows<GT> rg(a.gate, a.D, w0, rows, c, active);
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            Chan<GT, VEC> g;
            g.load(rg.r, rg.at(i));
            x[i].load(rx.r, rx.at(i));
            g.get(v[i]);
        }
    }
    const Borders bo = find_borders<TPT>(a, w0, end);
    RunDecay<KIND> A[VEC];
    float B[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) B[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if (__builtin_expect((bo.first >> i) & 1, 0)) load_state<VEC>(a.h0, bo.seq(i), a.D, c, B);
        float xv[VEC];
        x[i].get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float raw = v[i][e];
            v[i][e] = encode_gate<KIND>(raw);
            A[e].add(raw, v[i][e]);
            B[e] = step<KIND>(v[i][e], B[e], xv[e]);
            hide(v[i][e]);
            hide(B[e]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) sh.run[w][lane * VEC + e] = float2{bo.first ? kCut : A[e].get(), B[e]};
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        x[i].hide();
#pragma unroll
        for (int e = 0; e < VEC; ++e) hide(v[i][e]);
    }
    __syncthreads();
    chain<VEC, W, false>(a, sh, tile, c_tile);
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        h[e] = sh.carry[lane * VEC + e];
        if (w > 0) h[e] = apply_run(sh.run[w][lane * VEC + e], h[e]);
    }
    if (a.block_states && w0 % kLinearBlock == 0 && w0 < a.T) store_state<VEC>(a.block_states, w0 / kLinearBlock, a.D, c, h);
    const Rows<IO> ry(a.y, a.D, w0, rows, c, active);
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if (__builtin_expect((bo.first >> i) & 1, 0)) load_state<VEC>(a.h0, bo.seq(i), a.D, c, h);
        float xv[VEC];
        x[i].get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            h[e] = step<KIND>(v[i][e], h[e], xv[e]);
        Chan<IO, VEC>::put(ry.r, ry.at(i), h);
        __builtin_amdgcn_sched_barrier(0);
        if (__builtin_expect((bo.last >> i) & 1, 0)) store_state<VEC>(a.ht, bo.seq(i), a.D, c, h);
    }
    if (tile == 0) copy_empty<VEC, W>(a, a.h0, a.ht, c);
}

// =====================================================================================================
// backward.  The states are formed again from x and the tile's entering state (block_states); the carry
// c = a (dy + c') runs from the last token to the first, so the chain begins at the last tile.  x is as many
// bytes as y, and the states from it are not rounded to its type.  16384 x 4096 bf16, sigmoid: 151 us, 4.6 TB/s, VALU
// busy 60% of it with 51 instructions per element.
template <int KIND, typename IO, int VEC, int W, int TPT>
__global__ __launch_bounds__(64 * W, kWavesPerSimd) void linear_bwd_kernel(const LinearArgs a) {
    constexpr int L = W * TPT;
    static_assert(L % kLinearBlock == 0, "the workspace holds a word per channel and block, tiles begin at block states");
    __shared__ TileShared<VEC, W> sh;
    __shared__ float2 fwd[W][64 * VEC];
    const int64_t ticket = take_ticket(a, sh);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t place = ticket / a.nch, tile = a.tiles - 1 - place;
    const int64_t c_tile = (ticket % a.nch) * (64 * VEC);
    const int64_t c = c_tile + lane * VEC;
    const bool active = c < a.D;  // with VEC > 1 a lane's channels exist all or none
    const int64_t end = tokens_end(a);
    const int64_t w0 = tile * L + (int64_t)w * TPT;

    typedef typename GateT<KIND, IO>::T GT;
    const int rows = rows_of<TPT>(w0, end);
    Chan<IO, VEC> x[TPT], dy[TPT];
    float v[TPT][VEC];
    {
        const Rows<IO> rx(a.x, a.D, w0, rows, c, active), rdy(a.dy, a.D, w0, rows, c, active);
        const Rows<GT> rg(a.gate, a.D, w0, rows, c, active);
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            Chan<GT, VEC> g;
            g.load(rg.r, rg.at(i));
            x[i].load(rx.r, rx.at(i));
            dy[i].load(rdy.r, rdy.at(i));
            g.get(v[i]);
        }
    }
    const Borders bo = find_borders<TPT>(a, w0, end);
    auto hide_tile = [&] {
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
            x[i].hide();
            dy[i].hide();
#pragma unroll
            for (int e = 0; e < VEC; ++e) hide(v[i][e]);
        }
    };
    RunDecay<KIND> A[VEC];
    float B[VEC], C[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) B[e] = C[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if (__builtin_expect((bo.first >> i) & 1, 0)) load_state<VEC>(a.h0, bo.seq(i), a.D, c, B);
        float xv[VEC];
        x[i].get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float raw = v[i][e];
            v[i][e] = encode_gate<KIND>(raw);
            A[e].add(raw, v[i][e]);
            B[e] = step<KIND>(v[i][e], B[e], xv[e]);
            hide(v[i][e]);
            hide(B[e]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    hide_tile();
#pragma unroll
    for (int i = TPT - 1; i >= 0; --i) {
        if (__builtin_expect((bo.last >> i) & 1, 0)) load_state<VEC>(a.dht, bo.seq(i), a.D, c, C);
        float dv[VEC];
        dy[i].get(dv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            C[e] = mul_a(v[i][e], C[e] + dv[e]);
            hide(C[e]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const float decay = A[e].get();
        fwd[w][lane * VEC + e] = float2{bo.first ? kCut : decay, B[e]};
        sh.run[w][lane * VEC + e] = float2{bo.last ? kCut : decay, C[e]};
    }
    hide_tile();
    __syncthreads();
    chain<VEC, W, true>(a, sh, place, c_tile);
    float h[VEC], cr[VEC];
    load_state<VEC>(a.block_states, tile * (L / kLinearBlock), a.D, c, h);
    for (int i = 0; i < w; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = apply_run(fwd[i][lane * VEC + e], h[e]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        cr[e] = sh.carry[lane * VEC + e];
        if (w < W - 1) cr[e] = apply_run(sh.run[w][lane * VEC + e], cr[e]);
    }

    // dgate = D u: u holds a h_{t-1}, or a (1 - a) (h_{t-1} - x)
    float u[TPT][VEC];
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if (__builtin_expect((bo.first >> i) & 1, 0)) load_state<VEC>(a.h0, bo.seq(i), a.D, c, h);
        float xv[VEC];
        x[i].get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float vv = v[i][e], small = fabsf(vv);
            u[i][e] = KIND == kLogGate ? mul_a(vv, h[e]) : fmaf(-small, small, small) * (h[e] - xv[e]);
            h[e] = step<KIND>(vv, h[e], xv[e]);
            hide(u[i][e]);
            hide(h[e]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    hide_tile();
    const Rows<IO> rdx(a.dx, a.D, w0, rows, c, active);
    const Rows<GT> rdg(a.dgate, a.D, w0, rows, c, active);
#pragma unroll
    for (int i = TPT - 1; i >= 0; --i) {
        if (__builtin_expect((bo.last >> i) & 1, 0)) load_state<VEC>(a.dht, bo.seq(i), a.D, c, cr);
        float dv[VEC], dg[VEC];
        dy[i].get(dv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float Dt = dv[e] + cr[e];
            dg[e] = Dt * u[i][e];
            cr[e] = mul_a(v[i][e], Dt);
            dv[e] = KIND == kLogGate ? Dt : fmaf(v[i][e], Dt, near_one(v[i][e]) ? 0.0f : Dt);
        }
        Chan<IO, VEC>::put(rdx.r, rdx.at(i), dv);
        Chan<GT, VEC>::put(rdg.r, rdg.at(i), dg);
        __builtin_amdgcn_sched_barrier(0);
        if (__builtin_expect((bo.first >> i) & 1, 0)) store_state<VEC>(a.dh0, bo.seq(i), a.D, c, cr);
    }
    if (place == 0) copy_empty<VEC, W>(a, a.dht, a.dh0, c);
}

// All sequences empty: the final states are the initial ones, and so for the gradients.
__global__ __launch_bounds__(256) void linear_copy_kernel(const float* src, float* dst, int64_t count) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256)
        dst[i] = src ? src[i] : 0.0f;
}

// =====================================================================================================
// decode against a paged pool: one thread per (sequence, VEC channels).  The rows of AHEAD tokens are loaded
// together with the state, then computed in order: 4 where sequences may have more than one (64 sequences of 1 to
// 12 tokens, 4096 channels: 4.8 us, 7.0 with each token's rows loaded at its turn), else 1 (256 sequences: 3.9 us,
// 4.3 with the empty loads of 4).
template <int KIND, typename IO, typename ST, int VEC, int AHEAD>
__global__ __launch_bounds__(256) void linear_decode_kernel(const LinearArgs a) {
    const int n = blockIdx.y;
    const int slot = scalar_ints(a.slots)[n];
    if (slot < 0 || slot >= a.num_slots) return;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
    const bool active = c < a.D;
    int64_t bos = n, eos = n + 1;
    if (a.cu) {
        bos = scalar_ints(a.cu)[n];
        eos = scalar_ints(a.cu)[n + 1];
    }
    if (eos > a.T) eos = a.T;
    typedef typename GateT<KIND, IO>::T GT;
    const Rows<ST> rs(a.pool, a.D, slot, 1, c, active);
    Chan<ST, VEC> s;
    s.load(rs.r, rs.at(0));
    float h[VEC];
    for (int64_t t = bos; t < eos; t += AHEAD) {
        const int rows = eos - t < AHEAD ? (int)(eos - t) : AHEAD;
        const Rows<IO> rx(a.x, a.D, t, rows, c, active), ry(a.y, a.D, t, rows, c, active);
        const Rows<GT> rg(a.gate, a.D, t, rows, c, active);
        Chan<GT, VEC> g[AHEAD];
        Chan<IO, VEC> x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            g[i].load(rg.r, rg.at(i));
            x[i].load(rx.r, rx.at(i));
        }
        if (t == bos) s.get(h);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (i == rows) break;
            float gv[VEC], xv[VEC];
            g[i].get(gv);
            x[i].get(xv);
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[e] = step<KIND>(encode_gate<KIND>(gv[e]), h[e], xv[e]);
            Chan<IO, VEC>::put(ry.r, ry.at(i), h);
        }
    }
    if (a.commit && eos > bos) Chan<ST, VEC>::put(rs.r, rs.at(0), h);
}

template <int KIND, typename IO, int VEC, int W, int TPT, bool BACKWARD> hipError_t run_scan(LinearArgs a, hipStream_t s) {
    a.nch = (a.D + 64 * VEC - 1) / (64 * VEC);
    a.tiles = (a.T + W * TPT - 1) / (W * TPT);
    const int64_t blocks = a.tiles * a.nch;
    if (blocks >= (1ll << 32) / (64 * W)) return hipErrorInvalidValue;  // a launch has fewer than 2^32 threads
    if (a.tiles > 1) {
        const int64_t pairs = (a.tiles * a.D + 1) / 2;  // the workspace holds the word behind an odd count too
        linear_init_kernel<<<dim3((unsigned)((pairs + 255) / 256)), 256, 0, s>>>(a, pairs);
    }
    if constexpr (BACKWARD) linear_bwd_kernel<KIND, IO, VEC, W, TPT><<<dim3((unsigned)blocks), 64 * W, 0, s>>>(a);
    else linear_fwd_kernel<KIND, IO, VEC, W, TPT><<<dim3((unsigned)blocks), 64 * W, 0, s>>>(a);
    return hipGetLastError();
}

// VEC channels per lane need whole vectors: rows of a multiple of VEC channels, and aligned tensors.
bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <int KIND, typename IO, int VEC> bool vectors(const LinearArgs& a) {
    const int io = VEC * Elem<IO>::bytes, gt = VEC * Elem<typename GateT<KIND, IO>::T>::bytes;
    return a.D % VEC == 0 && aligned(a.x, io) && aligned(a.y, io) && aligned(a.dy, io) && aligned(a.dx, io) &&
           aligned(a.gate, gt) && aligned(a.dgate, gt);
}
constexpr int64_t kManyTiles = 128;

template <int KIND, typename IO, int VEC, int W, int TPT_FWD, int TPT_BWD>
hipError_t scan_tiles(const LinearArgs& a, bool backward, hipStream_t s) {
    return backward ? run_scan<KIND, IO, VEC, W, TPT_BWD, true>(a, s) : run_scan<KIND, IO, VEC, W, TPT_FWD, false>(a, s);
}

// Tiles (us of device time, log gate, bf16, forward; T x D).
//  - One tile needs no chain, and no launch before it.  Up to 64 tokens 8 per wave (64 x 1024: 5.7); to 128, 16; to
//    256, 16 waves of 16; to 512 the forward pass has 16 waves of 32.  One tile / what longer scans take, as replayed
//    in a graph, at 1024, 4096, 16384 and 65536 channels:
//      100 tokens  6.4 / 9.3    6.6 / 10.1   7.1 / 13.6   13.7 / 18.8, backward  8.5 / 10.7 and 22.0 / 16.7 at the ends
//      200 tokens  7.9 / 9.9    8.3 / 11.3   9.1 / 14.8   34.7 / 22.7, backward 10.9 / 11.6 and 50.3 / 48.1
//      333 tokens 12.3 / 10.4  12.7 / 12.1  13.9 / 21.4   56.5 / 53.9
//    (fp32 at 65536 channels 20 / 16, 39 / 44, 63 / 62).  Up to 16384 channels only 257 to 512 tokens of up to 4096
//    come out longer, by 3.1 at most; a call of its own saves more with the launch there (333 x 1024: 11.6 among
//    others, with a chain 14.4; 512 x 4096: 13.4 / 14.4).
//  - Chains of large tiles: two channels per lane; 32 tokens per wave in bf16, 16 in fp32 and in the bf16 backward
//    pass, whose kept values fill the registers.  The fp32 backward pass keeps 8: 16 spill (8192 x 4096: 143, 8
//    tokens 128).  Tiles of 4 or 16 waves were slower (32768 x 4096: 8 waves 207, 4 waves 219, 16 waves 247).
//  - Chains of small ones (8 tokens per wave) have more workgroups: large / small 333 x 4096 18.4 / 11.9,
//    2048 x 2048 20.5 / 22.4, 4096 x 2048 24.9 / 36.6: small below 128 large tiles.
//  - Odd rows go one channel per lane, 16 tokens per wave in their large tiles (333 x 515 10.7 / 9.4, 1000 x 515
//    11.9 / 12.0, 3001 x 515 16.3 / 21.2).
template <int KIND, typename IO> hipError_t scan(const LinearArgs& a, bool backward, hipStream_t s) {
    constexpr bool kHalf = Elem<IO>::bytes == 2;
    constexpr int F = kHalf ? 32 : 16, R = kHalf ? 16 : 8, W = 8;
    if (a.T > 64 && a.T <= 128) return scan_tiles<KIND, IO, 1, W, 16, 16>(a, backward, s);
    if (a.T > 128 && a.T <= 256) return scan_tiles<KIND, IO, 1, 16, 16, 16>(a, backward, s);
    if (!backward && a.T > 256 && a.T <= 512) return run_scan<KIND, IO, 1, 16, 32, false>(a, s);
    auto many = [&](int64_t tokens, int64_t channels) {
        return (a.T + tokens - 1) / tokens * ((a.D + channels - 1) / channels) >= kManyTiles;
    };
    if (vectors<KIND, IO, 2>(a))
        return many(W * (backward ? R : F), 128) ? scan_tiles<KIND, IO, 2, W, F, R>(a, backward, s)
                                                 : scan_tiles<KIND, IO, 2, W, 8, 8>(a, backward, s);
    return many(W * 16, 64) ? scan_tiles<KIND, IO, 1, W, 16, 16>(a, backward, s)
                            : scan_tiles<KIND, IO, 1, W, 8, 8>(a, backward, s);
}

template <int KIND, typename IO, typename ST, int VEC> hipError_t decode_run(const LinearArgs& a, hipStream_t s) {
    const int64_t per = 256 * VEC;
    const dim3 grid((unsigned)((a.D + per - 1) / per), (unsigned)a.N);
    if (a.max_q_len > 1) linear_decode_kernel<KIND, IO, ST, VEC, 4><<<grid, 256, 0, s>>>(a);
    else linear_decode_kernel<KIND, IO, ST, VEC, 1><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int KIND, typename IO, typename ST> hipError_t decode(const LinearArgs& a, hipStream_t s) {
    if (vectors<KIND, IO, 4>(a) && aligned(a.pool, 4 * Elem<ST>::bytes)) return decode_run<KIND, IO, ST, 4>(a, s);
    return decode_run<KIND, IO, ST, 1>(a, s);
}

template <int KIND, typename IO> hipError_t decode_st(const LinearArgs& a, int st_dtype, hipStream_t s) {
    return st_dtype == 0 ? decode<KIND, IO, float>(a, s) : decode<KIND, IO, bf16_t>(a, s);
}

}  // namespace

size_t linear_workspace(int64_t T, int64_t D) {
    const int64_t tiles = (T + kLinearBlock - 1) / kLinearBlock;
    return tiles > 1 ? 256 + ((size_t)tiles * (size_t)D + 1) * sizeof(uint64_t) : 0;  // the counter, the words
}

hipError_t launch_linear_scan(const LinearArgs& args, char* ws, int kind, int io_dtype, bool backward, hipStream_t s) {
    LinearArgs a = args;
    a.ticket = reinterpret_cast<uint32_t*>(ws);
    a.runs = reinterpret_cast<uint64_t*>(ws + 256);
    if (kind == kLogGate) return io_dtype == 0 ? scan<0, float>(a, backward, s) : scan<0, bf16_t>(a, backward, s);
    return io_dtype == 0 ? scan<1, float>(a, backward, s) : scan<1, bf16_t>(a, backward, s);
}

hipError_t launch_linear_copy(const float* src, float* dst, int64_t count, hipStream_t s) {
    const int64_t blocks = (count + 1023) / 1024;
    linear_copy_kernel<<<dim3((unsigned)(blocks < 2048 ? blocks : 2048)), 256, 0, s>>>(src, dst, count);
    return hipGetLastError();
}

hipError_t launch_linear_decode(const LinearArgs& a, int kind, int io_dtype, int st_dtype, hipStream_t s) {
    if (kind == kLogGate) return io_dtype == 0 ? decode_st<0, float>(a, st_dtype, s) : decode_st<0, bf16_t>(a, st_dtype, s);
    return io_dtype == 0 ? decode_st<1, float>(a, st_dtype, s) : decode_st<1, bf16_t>(a, st_dtype, s);
}

}  // namespace gdr
