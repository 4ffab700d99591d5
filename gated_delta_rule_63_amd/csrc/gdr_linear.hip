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
// Layout: a lane owns VEC neighbouring channels, a wave a run of TPT tokens, the 8 waves of a workgroup
// the 8 runs of a tile; a lane reads its channels' rows with one wide load each and walks them in time
// order in registers, so no value crosses lanes.
#include "gdr_device.h"
#include "gdr_internal.h"

namespace gdr {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kLogGate = 0;

// ---- a lane's VEC channels of one token, as loaded ----
template <typename T, int VEC> struct Chan;
template <typename T> struct Chan<T, 4> : RawVec<T, 4> {
    __device__ __forceinline__ static void put(void* p, int64_t i, const float* in) { Vec<T, 4>::store(p, i, in); }
};
template <typename T> struct Chan<T, 1> : RawElem<T> {
    __device__ __forceinline__ void get(float* out) const { out[0] = RawElem<T>::get(); }
    __device__ __forceinline__ static void put(void* p, int64_t i, const float* in) { Elem<T>::store(p, i, in[0]); }
};

template <int KIND, typename IO> struct GateT { typedef IO T; };
template <typename IO> struct GateT<kLogGate, IO> { typedef float T; };

// ---- gates ----
// A channel that forgets 1e-4 of its state per token needs that 1e-4 to more than the 2^-24 of 1 that a
// rounded a holds: the error repeats every token and would grow to 2^-24 / 1e-4 of the result.  A gate is
// therefore held as one float whose sign says which form it is: v = a - 1 <= -0 where a is near 1, v = a
// elsewhere, and a step adds the part that the rounded a lacks.
__device__ __forceinline__ float encode_gate_log(float g) {
    // -0.125 < g <= -0: e^g - 1 by its series (next term below 1e-9 of the result); +0 gives a = 1
    float p = fmaf(g, 1.0f / 720.0f, 1.0f / 120.0f);
    p = fmaf(g, p, 1.0f / 24.0f);
    p = fmaf(g, p, 1.0f / 6.0f);
    p = fmaf(g, p, 0.5f);
    p = fmaf(g, p, 1.0f);
    const uint32_t series = __float_as_uint(g * p) | 0x80000000u;
    const bool near_one = __float_as_uint(g) - 0x80000000u < 0x3E000000u;
    return near_one ? __uint_as_float(series) : exp_f32(g);
}

__device__ __forceinline__ float encode_gate_sigmoid(float z) {
    const float e = exp_f32(-fabsf(z));
    const float s = e * __builtin_amdgcn_rcpf(1.0f + e);  // the smaller of a and 1 - a
    return z >= 0.0f ? __uint_as_float(__float_as_uint(s) | 0x80000000u) : s;
}

template <int KIND> __device__ __forceinline__ float encode_gate(float raw) {
    return KIND == kLogGate ? encode_gate_log(raw) : encode_gate_sigmoid(raw);
}

__device__ __forceinline__ bool is_complement(float v) { return (int)__float_as_uint(v) < 0; }

struct Decay {
    float a, rest;  // a rounded, and what it lacks
    __device__ __forceinline__ explicit Decay(float v) {
        const bool c = is_complement(v);
        a = c ? 1.0f + v : v;
        rest = c ? v - (a - 1.0f) : 0.0f;
    }
    // a h + b; h is bounded in the correction so that an infinite h stays infinite
    __device__ __forceinline__ float step(float h, float b) const {
        const float hc = __builtin_amdgcn_fmed3f(h, -3.0e38f, 3.0e38f);
        return fmaf(a, h, fmaf(rest, hc, b));
    }
};

__device__ __forceinline__ float one_minus(float v) { return is_complement(v) ? -v : 1.0f - v; }

// ---- runs: (v, B), v the whole run's decay in the gates' form, or kCut ----
constexpr float kCut = __builtin_inff();

// The state behind a run entered with state h.
__device__ __forceinline__ float apply_run(float2 r, float h) { return r.x == kCut ? r.y : Decay(r.x).step(h, r.y); }

// 1 - A is kept where it is small and A where that is: a product of rounded decays near 1 would lose
// their complements as a single rounded decay does.
__device__ __forceinline__ float pick(float A, float Q) { return Q < 0.125f ? -Q : A; }

__device__ __forceinline__ float2 compose(float2 r1, float2 r2) {
    if (r2.x == kCut) return r2;
    const float B = Decay(r2.x).step(r1.y, r2.y);
    if (r1.x == kCut) return float2{kCut, B};
    const float q1 = one_minus(r1.x), q2 = one_minus(r2.x);
    return float2{pick(Decay(r1.x).a * Decay(r2.x).a, fmaf(q2, 1.0f - q1, q1)), B};
}

// The decay of a run of gates: the log gates' sum, or the product of the decays beside its complement.
template <int KIND> struct RunDecay;
template <> struct RunDecay<kLogGate> {
    float G = 0.0f;
    __device__ __forceinline__ void add(float raw, float) { G += raw; }
    __device__ __forceinline__ float get() const { return encode_gate_log(G); }
};
template <> struct RunDecay<1> {
    float A = 1.0f, Q = 0.0f;
    __device__ __forceinline__ void add(float, float v) {
        const Decay d(v);
        A = fmaf(d.a, A, d.rest * A);
        Q = fmaf(one_minus(v), 1.0f - Q, Q);
    }
    __device__ __forceinline__ float get() const { return pick(A, Q); }
};

// ---- which of a wave's TPT tokens begin and end a sequence ----
struct Borders {
    uint64_t first, last;  // bit i: token w0 + i is the first / last of its sequence
    int n;                 // lane i: the sequence of token w0 + i
    __device__ __forceinline__ int seq(int i) const { return __builtin_amdgcn_readlane(n, i); }
};

__device__ __forceinline__ int64_t tokens_end(const LinearArgs& a) {
    if (!a.cu) return a.T;
    const int64_t e = a.cu[a.N];
    return e < a.T ? e : a.T;
}

template <int TPT> __device__ __forceinline__ Borders find_borders(const LinearArgs& a, int64_t w0, int64_t end) {
    static_assert(TPT <= 64, "one lane per token");
    Borders b;
    const int lane = threadIdx.x & 63;
    const int64_t t = w0 + lane;
    const bool in = lane < TPT && t < end;
    if (!a.cu) {
        b.n = 0;
        b.first = __ballot(in && t == 0);
        b.last = __ballot(in && t == end - 1);
        return b;
    }
    int lo = 0, hi = a.N;  // the last n < N with cu[n] <= t: empty sequences at t come before it
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= t) lo = mid; else hi = mid;
    }
    b.n = lo;
    b.first = __ballot(in && a.cu[lo] == t);
    b.last = __ballot(in && a.cu[lo + 1] == t + 1);
    return b;
}

__device__ __forceinline__ float2* run_word(const LinearArgs& a, int64_t tile, int64_t c) {
    return a.runs + tile * a.D + c;
}

template <int VEC> __device__ __forceinline__ void load_state(const float* p, int64_t i, float* out) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = p ? p[i + e] : 0.0f;
}
template <int VEC> __device__ __forceinline__ void store_state(float* p, int64_t i, const float* in) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) p[i + e] = in[e];
}

// Writes the tile's run: each channel's 8 waves composed in the order FIRST .. LAST.
template <int VEC, bool REVERSE>
__device__ __forceinline__ void publish_run(const LinearArgs& a, const float2 (*run)[64 * VEC], int64_t tile, int64_t c_tile) {
    for (int c = threadIdx.x; c < 64 * VEC; c += kThreads) {
        if (c_tile + c >= a.D) continue;
        float2 r = run[REVERSE ? kWaves - 1 : 0][c];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) r = compose(r, run[REVERSE ? kWaves - 1 - i : i][c]);
        *run_word(a, tile, c_tile + c) = r;
    }
}

// =====================================================================================================
// forward.  APPLY false: only the tile's run is written; true: the tile's entering state is read from the
// same word, and outputs, final states and block states are written.
template <int KIND, typename IO, int VEC, int TPT, bool APPLY>
__global__ __launch_bounds__(kThreads) void linear_fwd_kernel(const LinearArgs a) {
    constexpr int L = kWaves * TPT;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tile = blockIdx.x / a.nch;
    const int64_t c_tile = (int64_t)(blockIdx.x % a.nch) * (64 * VEC);
    const int64_t c = c_tile + lane * VEC;
    const bool active = c < a.D;
    const int64_t end = tokens_end(a);
    const int64_t w0 = tile * L + (int64_t)w * TPT;
    const Borders bo = find_borders<TPT>(a, w0, end);

    typedef typename GateT<KIND, IO>::T GT;
    __shared__ float2 run[kWaves][64 * VEC];
    Chan<IO, VEC> x[TPT];
    float v[TPT][VEC];
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const bool in = active && w0 + i < end;
        const int64_t at = (w0 + i) * a.D + c;
        Chan<GT, VEC> g{};
        x[i] = Chan<IO, VEC>{};
        if (in) {
            g.load(a.gate, at);
            x[i].load(a.x, at);
        }
        g.get(v[i]);
    }
    RunDecay<KIND> A[VEC];
    float B[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) B[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if ((bo.first >> i) & 1) {
            if (active) load_state<VEC>(a.h0, (int64_t)bo.seq(i) * a.D + c, B);
        }
        float xv[VEC];
        x[i].get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float raw = v[i][e];
            v[i][e] = encode_gate<KIND>(raw);
            A[e].add(raw, v[i][e]);
            B[e] = Decay(v[i][e]).step(B[e], KIND == kLogGate ? xv[e] : one_minus(v[i][e]) * xv[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) run[w][lane * VEC + e] = float2{bo.first ? kCut : A[e].get(), B[e]};
    __syncthreads();
    if constexpr (!APPLY) {
        publish_run<VEC, false>(a, run, tile, c_tile);
        return;
    }
    if (!active) return;
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = tile > 0 ? run_word(a, tile, c + e)->y : 0.0f;
    for (int i = 0; i < w; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = apply_run(run[i][lane * VEC + e], h[e]);
    if (a.block_states && w0 % kLinearBlock == 0 && w0 < a.T) store_state<VEC>(a.block_states, w0 / kLinearBlock * a.D + c, h);
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if (w0 + i >= end) break;
        if ((bo.first >> i) & 1) load_state<VEC>(a.h0, (int64_t)bo.seq(i) * a.D + c, h);
        float xv[VEC];
        x[i].get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            h[e] = Decay(v[i][e]).step(h[e], KIND == kLogGate ? xv[e] : one_minus(v[i][e]) * xv[e]);
        Chan<IO, VEC>::put(a.y, (w0 + i) * a.D + c, h);
        if (((bo.last >> i) & 1) && a.ht) store_state<VEC>(a.ht, (int64_t)bo.seq(i) * a.D + c, h);
    }
}

// =====================================================================================================
// backward.  The states are formed again from x and the tile's entering state (block_states); the carry
// c = a (dy + c') runs from the last token to the first.
template <int KIND, typename IO, int VEC, int TPT, bool APPLY>
__global__ __launch_bounds__(kThreads) void linear_bwd_kernel(const LinearArgs a) {
    constexpr int L = kWaves * TPT;
    static_assert(L % kLinearBlock == 0, "a tile begins at a block state");
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tile = blockIdx.x / a.nch;
    const int64_t c_tile = (int64_t)(blockIdx.x % a.nch) * (64 * VEC);
    const int64_t c = c_tile + lane * VEC;
    const bool active = c < a.D;
    const int64_t end = tokens_end(a);
    const int64_t w0 = tile * L + (int64_t)w * TPT;
    const Borders bo = find_borders<TPT>(a, w0, end);

    typedef typename GateT<KIND, IO>::T GT;
    __shared__ float2 fwd[kWaves][64 * VEC], rev[kWaves][64 * VEC];
    Chan<IO, VEC> x[TPT], dy[TPT];
    float v[TPT][VEC];
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        const bool in = active && w0 + i < end;
        const int64_t at = (w0 + i) * a.D + c;
        Chan<GT, VEC> g{};
        x[i] = Chan<IO, VEC>{};
        dy[i] = Chan<IO, VEC>{};
        if (in) {
            g.load(a.gate, at);
            dy[i].load(a.dy, at);
            if constexpr (APPLY) x[i].load(a.x, at);
        }
        g.get(v[i]);
    }
    RunDecay<KIND> A[VEC];
    float B[VEC], C[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) B[e] = C[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if ((bo.first >> i) & 1) {
            if (APPLY && active) load_state<VEC>(a.h0, (int64_t)bo.seq(i) * a.D + c, B);
        }
        float xv[VEC];
        x[i].get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float raw = v[i][e];
            v[i][e] = encode_gate<KIND>(raw);
            A[e].add(raw, v[i][e]);
            if constexpr (APPLY) B[e] = Decay(v[i][e]).step(B[e], KIND == kLogGate ? xv[e] : one_minus(v[i][e]) * xv[e]);
        }
    }
#pragma unroll
    for (int i = TPT - 1; i >= 0; --i) {
        if ((bo.last >> i) & 1) {
            if (active) load_state<VEC>(a.dht, (int64_t)bo.seq(i) * a.D + c, C);
        }
        float dv[VEC];
        dy[i].get(dv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) C[e] = Decay(v[i][e]).step(C[e] + dv[e], 0.0f);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const float decay = A[e].get();
        if constexpr (APPLY) fwd[w][lane * VEC + e] = float2{bo.first ? kCut : decay, B[e]};
        rev[w][lane * VEC + e] = float2{bo.last ? kCut : decay, C[e]};
    }
    __syncthreads();
    if constexpr (!APPLY) {
        publish_run<VEC, true>(a, rev, tile, c_tile);
        return;
    }
    if (!active) return;
    float h[VEC], cr[VEC];
    load_state<VEC>(a.block_states, tile * (L / kLinearBlock) * a.D + c, h);
#pragma unroll
    for (int e = 0; e < VEC; ++e) cr[e] = tile + 1 < a.tiles ? run_word(a, tile, c + e)->y : 0.0f;
    for (int i = 0; i < w; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = apply_run(fwd[i][lane * VEC + e], h[e]);
    for (int i = kWaves - 1; i > w; --i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) cr[e] = apply_run(rev[i][lane * VEC + e], cr[e]);

    // dgate = D u: u holds a h_{t-1}, or a (1 - a) (h_{t-1} - x)
    float u[TPT][VEC];
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
        if ((bo.first >> i) & 1) load_state<VEC>(a.h0, (int64_t)bo.seq(i) * a.D + c, h);
        float xv[VEC];
        x[i].get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const Decay d(v[i][e]);
            const float q = one_minus(v[i][e]);
            u[i][e] = KIND == kLogGate ? d.a * h[e] : d.a * q * (h[e] - xv[e]);
            h[e] = d.step(h[e], KIND == kLogGate ? xv[e] : q * xv[e]);
        }
    }
#pragma unroll
    for (int i = TPT - 1; i >= 0; --i) {
        if (w0 + i >= end) continue;
        if ((bo.last >> i) & 1) load_state<VEC>(a.dht, (int64_t)bo.seq(i) * a.D + c, cr);
        float dv[VEC], dg[VEC];
        dy[i].get(dv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float Dt = dv[e] + cr[e];
            dg[e] = Dt * u[i][e];
            cr[e] = Decay(v[i][e]).step(Dt, 0.0f);
            dv[e] = KIND == kLogGate ? Dt : one_minus(v[i][e]) * Dt;
        }
        const int64_t at = (w0 + i) * a.D + c;
        Chan<IO, VEC>::put(a.dx, at, dv);
        Chan<GT, VEC>::put(a.dgate, at, dg);
        if (((bo.first >> i) & 1) && a.dh0) store_state<VEC>(a.dh0, (int64_t)bo.seq(i) * a.D + c, cr);
    }
}

// Turns every tile's run into the state that enters it, tile by tile (from the last for the backward pass).
template <bool REVERSE> __global__ __launch_bounds__(64) void linear_carry_kernel(const LinearArgs a) {
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (c >= a.D) return;
    float h = 0.0f;
    for (int64_t i = 0; i < a.tiles; ++i) {
        float2* word = run_word(a, REVERSE ? a.tiles - 1 - i : i, c);
        const float2 r = *word;
        *word = float2{0.0f, h};
        h = apply_run(r, h);
    }
}

// Empty sequences: the final state is the initial one, and so for the gradients.
__global__ __launch_bounds__(256) void linear_empty_kernel(const int32_t* cu, const float* src, float* dst, int64_t D) {
    const int64_t n = blockIdx.y;
    if (cu && cu[n + 1] != cu[n]) return;
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < D; c += (int64_t)gridDim.x * 256)
        dst[n * D + c] = src ? src[n * D + c] : 0.0f;
}

// =====================================================================================================
// decode against a paged pool: one thread per (sequence, VEC channels)
template <int KIND, typename IO, typename ST, int VEC>
__global__ __launch_bounds__(256) void linear_decode_kernel(const LinearArgs a) {
    const int n = blockIdx.y;
    const int slot = a.slots[n];
    if (slot < 0 || slot >= a.num_slots) return;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
    if (c >= a.D) return;
    const int64_t bos = a.cu ? a.cu[n] : n;
    int64_t eos = a.cu ? a.cu[n + 1] : n + 1;
    if (eos > a.T) eos = a.T;
    typedef typename GateT<KIND, IO>::T GT;
    Chan<ST, VEC> s;
    s.load(a.pool, (int64_t)slot * a.D + c);
    float h[VEC];
    s.get(h);
    for (int64_t t = bos; t < eos; ++t) {
        Chan<GT, VEC> g;
        Chan<IO, VEC> x;
        g.load(a.gate, t * a.D + c);
        x.load(a.x, t * a.D + c);
        float gv[VEC], xv[VEC];
        g.get(gv);
        x.get(xv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float v = encode_gate<KIND>(gv[e]);
            h[e] = Decay(v).step(h[e], KIND == kLogGate ? xv[e] : one_minus(v) * xv[e]);
        }
        Chan<IO, VEC>::put(a.y, t * a.D + c, h);
    }
    if (a.commit) Chan<ST, VEC>::put(a.pool, (int64_t)slot * a.D + c, h);
}

template <int KIND, typename IO, int VEC, int TPT> hipError_t run_fwd(LinearArgs a, hipStream_t s) {
    a.nch = (a.D + 64 * VEC - 1) / (64 * VEC);
    a.tiles = (a.T + kWaves * TPT - 1) / (kWaves * TPT);
    const int64_t blocks = a.tiles * a.nch;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (a.tiles > 1) {
        linear_fwd_kernel<KIND, IO, VEC, TPT, false><<<dim3((unsigned)blocks), kThreads, 0, s>>>(a);
        linear_carry_kernel<false><<<dim3((unsigned)((a.D + 63) / 64)), 64, 0, s>>>(a);
    }
    linear_fwd_kernel<KIND, IO, VEC, TPT, true><<<dim3((unsigned)blocks), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <int KIND, typename IO, int VEC, int TPT> hipError_t run_bwd(LinearArgs a, hipStream_t s) {
    a.nch = (a.D + 64 * VEC - 1) / (64 * VEC);
    a.tiles = (a.T + kWaves * TPT - 1) / (kWaves * TPT);
    const int64_t blocks = a.tiles * a.nch;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (a.tiles > 1) {
        linear_bwd_kernel<KIND, IO, VEC, TPT, false><<<dim3((unsigned)blocks), kThreads, 0, s>>>(a);
        linear_carry_kernel<true><<<dim3((unsigned)((a.D + 63) / 64)), 64, 0, s>>>(a);
    }
    linear_bwd_kernel<KIND, IO, VEC, TPT, true><<<dim3((unsigned)blocks), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

// Four channels per lane need whole vectors: rows of a multiple of four channels, and aligned tensors.
bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

template <int KIND, typename IO> bool wide_ok(const LinearArgs& a) {
    const int io = 4 * Elem<IO>::bytes, gt = 4 * Elem<typename GateT<KIND, IO>::T>::bytes;
    return a.D % 4 == 0 && aligned(a.x, io) && aligned(a.y, io) && aligned(a.dy, io) && aligned(a.dx, io) &&
           aligned(a.gate, gt) && aligned(a.dgate, gt);
}

template <int KIND, typename IO> hipError_t scan(const LinearArgs& a, bool backward, hipStream_t s) {
    if (wide_ok<KIND, IO>(a)) return backward ? run_bwd<KIND, IO, 4, 8>(a, s) : run_fwd<KIND, IO, 4, 8>(a, s);
    return backward ? run_bwd<KIND, IO, 1, 8>(a, s) : run_fwd<KIND, IO, 1, 8>(a, s);
}

template <int KIND, typename IO, typename ST, int VEC> hipError_t decode_run(const LinearArgs& a, hipStream_t s) {
    const int64_t per = 256 * VEC;
    linear_decode_kernel<KIND, IO, ST, VEC><<<dim3((unsigned)((a.D + per - 1) / per), (unsigned)a.N), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int KIND, typename IO, typename ST> hipError_t decode(const LinearArgs& a, hipStream_t s) {
    if (wide_ok<KIND, IO>(a) && aligned(a.pool, 4 * Elem<ST>::bytes)) return decode_run<KIND, IO, ST, 4>(a, s);
    return decode_run<KIND, IO, ST, 1>(a, s);
}

template <int KIND, typename IO> hipError_t decode_st(const LinearArgs& a, int st_dtype, hipStream_t s) {
    return st_dtype == 0 ? decode<KIND, IO, float>(a, s) : decode<KIND, IO, bf16_t>(a, s);
}

}  // namespace

size_t linear_workspace(int64_t T, int64_t D) {
    const int64_t tiles = (T + kLinearBlock - 1) / kLinearBlock;
    return tiles > 1 ? (size_t)tiles * (size_t)D * sizeof(float2) : 0;
}

hipError_t launch_linear_scan(const LinearArgs& a, int kind, int io_dtype, bool backward, hipStream_t s) {
    hipError_t e;
    if (kind == kLogGate) e = io_dtype == 0 ? scan<0, float>(a, backward, s) : scan<0, bf16_t>(a, backward, s);
    else e = io_dtype == 0 ? scan<1, float>(a, backward, s) : scan<1, bf16_t>(a, backward, s);
    if (e != hipSuccess) return e;
    float* dst = backward ? a.dh0 : a.ht;
    if (!a.cu || !dst) return hipSuccess;
    return launch_linear_empty(a.cu, backward ? a.dht : a.h0, dst, a.N, a.D, s);
}

hipError_t launch_linear_empty(const int32_t* cu, const float* src, float* dst, int32_t N, int64_t D, hipStream_t s) {
    const unsigned nx = (unsigned)((D + 255) / 256 < 64 ? (D + 255) / 256 : 64);
    linear_empty_kernel<<<dim3(nx, (unsigned)N), 256, 0, s>>>(cu, src, dst, D);
    return hipGetLastError();
}

hipError_t launch_linear_decode(const LinearArgs& a, int kind, int io_dtype, int st_dtype, hipStream_t s) {
    if (kind == kLogGate) return io_dtype == 0 ? decode_st<0, float>(a, st_dtype, s) : decode_st<0, bf16_t>(a, st_dtype, s);
    return io_dtype == 0 ? decode_st<1, float>(a, st_dtype, s) : decode_st<1, bf16_t>(a, st_dtype, s);
}

}  // namespace gdr
