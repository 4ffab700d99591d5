// Rotary positions applied to q and k, and k and v written into the pages of a cache (gdr_rope_append_paged).
//
// A pair (x, y) at position p turns by theta = sum_a p_a f_a: (x cos - y sin, y cos + x sin).  The angle is formed
// and reduced to turns in 64 bits: at position 10^6 a 32-bit product would already be off by 0.03 radians.
// A workgroup takes one token and all its heads, forms each pair's cosine and sine once into the LDS, and then only
// moves data: two 16-byte pieces per thread, the pair's halves, so that a row may be rotated in place.
//
// HBM bounds it: 32768 bf16 tokens of 32 + 8 + 8 heads of 128 channels, 403 MB read and 470 written, take 144 us (6.0
// TB/s; a large copy reaches 4.95).  With 8, 4 and 2 tokens per workgroup it was 163, 158 and 147: the angles of one token
// are formed while others' rows move.  256 tokens take 5 us: the launch and one chain of dependent loads, of which a binary
// search for the token's sequence is eight, then its context, its page and its row.  Pairs of halves whose number does not
// fill 16-byte pieces go one element at a time: with 34 of 128 channels rotated the 32768 tokens take 297 us.
#include <hip/hip_runtime.h>

#include "gdr_attn_device.h"

namespace gdr {
namespace {

constexpr int64_t kTokens = 1 << 22;   // of a launch, at most: it has fewer than 2^32 threads
// Bytes moved, past what the last cache holds, from which on rows are read and written past the caches: 872 MB 154 us
// through them and 146 past them, 436 MB 79 and 74; 218 MB 36 and 39, 215 MB of fp32 40 and 47.
constexpr int64_t kLarge = (int64_t)1 << 28;

// NT: rows of a large batch are read and written past the caches.
template <bool NT> __device__ __forceinline__ u32x4_t read16(const char* p, int c) {
    const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p) + c;
    if constexpr (NT) return __builtin_nontemporal_load(q);
    return *q;
}
template <bool NT> __device__ __forceinline__ void write16(char* p, int c, const u32x4_t& x) {
    u32x4_t* q = reinterpret_cast<u32x4_t*>(p) + c;
    if constexpr (NT) __builtin_nontemporal_store(x, q);
    else *q = x;
}

template <typename T, int D, int MODE, bool NT>  // MODE 0: pairs (i, i + R/2) in 16-byte pieces; 1: pairs (2i, 2i + 1); 2: (i, i + R/2), any R
__global__ __launch_bounds__(512) void rope_append_kernel(RopeArgs a) {
    constexpr int es = Elem<T>::bytes, V = 16 / es, units = MODE == 2 ? D / 2 : D / V / 2;
    __shared__ float cj[D / 2], sj[D / 2];
    const int64_t t = a.first + blockIdx.x;
    const int half = a.rotary / 2;
    int n = 0, first = 0;
    if (a.cu) {
        if (t >= a.cu[a.N]) return;
        n = find_seq(a.cu, a.N, (int)t);
        first = a.cu[n];
    } else if (a.one_token) {
        first = n = (int)t;
    }
    const int ctx = a.context ? a.context[n] : 0;
    if (ctx < 0) return;
    const int64_t place = (int64_t)ctx + (t - first);   // in the cache, and in the sequence
    int page_id = -1;
    const int row = (int)(place & ((1 << a.page_shift) - 1));
    if (a.k_pages && (place >> a.page_shift) < a.max_pages) {
        page_id = a.table[(int64_t)n * a.max_pages + (place >> a.page_shift)];
        if (page_id >= a.num_pages) page_id = -1;
    }
    for (int p = threadIdx.x; p < half; p += blockDim.x) {
        double theta = 0.0;
        if (a.positions) {
            for (int x = 0; x < a.axes; ++x) theta += (double)a.positions[x * a.T + t] * (double)a.freq[x * half + p];
        } else {
            theta = (double)place * (double)a.freq[p];
        }
        // whole turns off, 2 pi in two parts
        const double turns = rint(theta * 0.15915494309189535);
        const double rest = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, theta));
        double s, c;
        sincospi(rest * 0.3183098861837907, &s, &c);
        cj[p] = (float)c;
        sj[p] = (float)s;
    }
    __syncthreads();
    const int all = (a.HQ + 2 * a.HK) * units;
    for (int i = threadIdx.x; i < all; i += blockDim.x) {
        const int h = i / units, u = i % units;
        const int kind = h < a.HQ ? 0 : h < a.HQ + a.HK ? 1 : 2;
        const int hh = kind == 0 ? h : kind == 1 ? h - a.HQ : h - a.HQ - a.HK;
        const char* src;
        char *dst = nullptr, *page = nullptr;
        const int64_t at = (((int64_t)page_id * a.HK + hh) << a.page_shift) + row;
        if (kind == 0) {
            if (!a.q) continue;
            src = static_cast<const char*>(a.q) + (t * a.q_stride + (int64_t)hh * D) * es;
            dst = static_cast<char*>(a.q_out) + (t * a.HQ + hh) * D * es;
        } else if (kind == 1) {
            src = static_cast<const char*>(a.k) + (t * a.k_stride + (int64_t)hh * D) * es;
            if (a.k_out) dst = static_cast<char*>(a.k_out) + (t * a.HK + hh) * D * es;
            if (page_id >= 0) page = static_cast<char*>(a.k_pages) + at * D * es;
        } else {
            if (page_id < 0) continue;
            src = static_cast<const char*>(a.v) + (t * a.v_stride + (int64_t)hh * D) * es;
            page = static_cast<char*>(a.v_pages) + at * D * es;
        }
        if constexpr (MODE == 2) {
            // pair u, or two channels behind the rotated ones
            const bool turn = u < half;
            const int c0 = turn ? u : 2 * half + 2 * (u - half), c1 = turn ? u + half : c0 + 1;
            float x = Elem<T>::load(src, c0), y = Elem<T>::load(src, c1);
            if (kind < 2 && turn) {
                const float c = cj[u], s = sj[u], z = x * c - y * s;
                y = y * c + x * s;
                x = z;
            }
            if (dst) { Elem<T>::store(dst, c0, x); Elem<T>::store(dst, c1, y); }
            if (page) { Elem<T>::store(page, c0, x); Elem<T>::store(page, c1, y); }
        } else {
            const int rot = MODE == 0 ? half / V : 0;   // pieces that hold first halves of pairs
            const int c0 = MODE == 0 && u < rot ? u : MODE == 0 ? 2 * rot + 2 * (u - rot) : 2 * u;
            const int c1 = MODE == 0 && u < rot ? u + rot : c0 + 1;
            u32x4_t raw0 = read16<NT>(src, c0), raw1 = read16<NT>(src, c1);
            if (kind < 2 && (MODE == 0 ? u < rot : 2 * V * u < a.rotary)) {
                float x[V], y[V];
                Vec<T, V>::load(&raw0, 0, x);
                Vec<T, V>::load(&raw1, 0, y);
                if constexpr (MODE == 0) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float c = cj[V * u + e], s = sj[V * u + e], z = x[e] * c - y[e] * s;
                        y[e] = y[e] * c + x[e] * s;
                        x[e] = z;
                    }
                } else {
                    auto turn = [&](float* v, int first) {
#pragma unroll
                        for (int e = 0; e < V / 2; ++e) {
                            const int p = first + e;
                            if (p < half) {
                                const float c = cj[p], s = sj[p], z = v[2 * e] * c - v[2 * e + 1] * s;
                                v[2 * e + 1] = v[2 * e + 1] * c + v[2 * e] * s;
                                v[2 * e] = z;
                            }
                        }
                    };
                    turn(x, V * u);
                    turn(y, V * u + V / 2);
                }
                Vec<T, V>::store(&raw0, 0, x);
                Vec<T, V>::store(&raw1, 0, y);
            }
            if (dst) { write16<NT>(dst, c0, raw0); write16<NT>(dst, c1, raw1); }
            if (page) { write16<NT>(page, c0, raw0); write16<NT>(page, c1, raw1); }
        }
    }
}

template <typename T, int D, bool NT>
hipError_t launch(const RopeArgs& a, hipStream_t stream) {
    constexpr int V = 16 / Elem<T>::bytes;
    const dim3 grid((unsigned)min(a.T - a.first, kTokens));
    // a thread per piece of the token where that is at most eight waves
    const int64_t pieces = (int64_t)(a.HQ + 2 * a.HK) * (D / V / 2);
    const int threads = (int)min((int64_t)512, (pieces + 63) / 64 * 64);
    if (a.interleaved) rope_append_kernel<T, D, 1, NT><<<grid, threads, 0, stream>>>(a);
    else if (a.rotary / 2 % V == 0) rope_append_kernel<T, D, 0, NT><<<grid, threads, 0, stream>>>(a);
    else rope_append_kernel<T, D, 2, false><<<grid, 512, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch(const RopeArgs& a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    const bool large = a.T * (2 * a.HQ + 5 * a.HK) * D * Elem<T>::bytes >= kLarge;
    for (RopeArgs part = a; part.first < a.T && e == hipSuccess; part.first += kTokens)
        e = large ? launch<T, D, true>(part, stream) : launch<T, D, false>(part, stream);
    return e;
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, int D, int io_dtype, hipStream_t stream) {
    if (io_dtype == 1) return D == 64 ? launch<bf16_t, 64>(a, stream) : launch<bf16_t, 128>(a, stream);
    return D == 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace gdr
