// Rotary positions applied to q and k, and k and v written into the pages of a cache (gdr_rope_append_paged).
//
// A pair (x, y) at position p turns by theta = sum_a p_a f_a: (x cos - y sin, y cos + x sin).  The angle is formed
// and reduced to turns in 64 bits: at position 10^6 a 32-bit product would already be off by 0.03 radians.
// A workgroup takes a few tokens and all their heads, forms each (token, pair)'s cosine and sine once into the
// LDS, and then only moves data: two 16-byte pieces per thread and step, the pair's halves, so that a row may be
// rotated in place.
#include <hip/hip_runtime.h>

#include "gdr_attn_device.h"

namespace gdr {
namespace {

constexpr int kMaxTokens = 8;   // tokens per workgroup at most

// Places of one token: where its row of the cache is, and whether it takes part at all.
struct RopeToken {
    int live;        // 0: padded sequence, or a row behind the last one
    int page, row;   // page < 0: no page for it
    int pos;         // context + index in the sequence
};

template <typename T, int D, int MODE>  // MODE 0: pairs (i, i + R/2) in 16-byte pieces; 1: pairs (2i, 2i + 1); 2: (i, i + R/2), any R
__global__ __launch_bounds__(256) void rope_append_kernel(RopeArgs a) {
    constexpr int es = Elem<T>::bytes, V = 16 / es, units = MODE == 2 ? D / 2 : D / V / 2;
    __shared__ RopeToken tok[kMaxTokens];
    __shared__ float cs[kMaxTokens * D / 2], sn[kMaxTokens * D / 2];
    const int64_t t0 = (int64_t)blockIdx.x * a.per;
    const int tid = threadIdx.x, half = a.rotary / 2;
    const int count = (int)min((int64_t)a.per, a.T - t0);
    if (tid < count) {
        const int64_t t = t0 + tid;
        RopeToken k;
        int n, first;
        if (a.cu) {
            n = find_seq(a.cu, a.N, (int)t);
            first = a.cu[n];
            k.live = t < a.cu[a.N];
        } else {
            n = a.one_token ? (int)t : 0;
            first = n;
            k.live = 1;
        }
        const int ctx = a.context ? a.context[n] : 0;
        if (ctx < 0) k.live = 0;
        const int64_t at = (int64_t)ctx + (t - first);
        k.pos = (int)at;
        k.page = -1;
        k.row = 0;
        if (a.k_pages && k.live) {
            const int64_t i = at >> a.page_shift;
            k.row = (int)(at & ((1 << a.page_shift) - 1));
            if (i < a.max_pages) {
                const int p = a.table[(int64_t)n * a.max_pages + i];
                if (p >= 0 && p < a.num_pages) k.page = p;
            }
        }
        tok[tid] = k;
    }
    __syncthreads();
    for (int i = tid; i < count * half; i += 256) {
        const int j = i / half, p = i % half;
        double theta = 0.0;
        if (a.positions) {
            for (int x = 0; x < a.axes; ++x) theta += (double)a.positions[x * a.T + t0 + j] * (double)a.freq[x * half + p];
        } else {
            theta = (double)tok[j].pos * (double)a.freq[p];
        }
        // whole turns off, 2 pi in two parts
        const double turns = rint(theta * 0.15915494309189535);
        const double rest = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, theta));
        double s, c;
        sincospi(rest * 0.3183098861837907, &s, &c);
        cs[j * (D / 2) + p] = (float)c;
        sn[j * (D / 2) + p] = (float)s;
    }
    __syncthreads();
    const int heads = a.HQ + 2 * a.HK, per_token = heads * units;
    for (int i = tid; i < count * per_token; i += 256) {
        const int j = i / per_token, r = i % per_token, h = r / units, u = r % units;
        const RopeToken k = tok[j];
        if (!k.live) continue;
        const int64_t t = t0 + j;
        const int kind = h < a.HQ ? 0 : h < a.HQ + a.HK ? 1 : 2;
        const int hh = kind == 0 ? h : kind == 1 ? h - a.HQ : h - a.HQ - a.HK;
        const char* src;
        char *dst, *page = nullptr;
        const int64_t at = (((int64_t)k.page * a.HK + hh) << a.page_shift) + k.row;
        if (kind == 0) {
            if (!a.q) continue;
            src = static_cast<const char*>(a.q) + (t * a.q_stride + (int64_t)hh * D) * es;
            dst = static_cast<char*>(a.q_out) + (t * a.HQ + hh) * D * es;
        } else if (kind == 1) {
            src = static_cast<const char*>(a.k) + (t * a.k_stride + (int64_t)hh * D) * es;
            dst = a.k_out ? static_cast<char*>(a.k_out) + (t * a.HK + hh) * D * es : nullptr;
            if (k.page >= 0) page = static_cast<char*>(a.k_pages) + at * D * es;
        } else {
            if (k.page < 0) continue;
            src = static_cast<const char*>(a.v) + (t * a.v_stride + (int64_t)hh * D) * es;
            dst = nullptr;
            page = static_cast<char*>(a.v_pages) + at * D * es;
        }
        const float *cj = cs + j * (D / 2), *sj = sn + j * (D / 2);
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
            uint4 raw0 = reinterpret_cast<const uint4*>(src)[c0], raw1 = reinterpret_cast<const uint4*>(src)[c1];
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
            if (dst) { reinterpret_cast<uint4*>(dst)[c0] = raw0; reinterpret_cast<uint4*>(dst)[c1] = raw1; }
            if (page) { reinterpret_cast<uint4*>(page)[c0] = raw0; reinterpret_cast<uint4*>(page)[c1] = raw1; }
        }
    }
}

template <typename T, int D>
hipError_t launch(const RopeArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.T + a.per - 1) / a.per));
    constexpr int V = 16 / Elem<T>::bytes;
    if (a.interleaved) rope_append_kernel<T, D, 1><<<grid, 256, 0, stream>>>(a);
    else if (a.rotary / 2 % V == 0) rope_append_kernel<T, D, 0><<<grid, 256, 0, stream>>>(a);
    else rope_append_kernel<T, D, 2><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_append(RopeArgs a, int D, int io_dtype, hipStream_t stream) {
    a.per = a.T >= 4096 ? kMaxTokens : 1;
    if (io_dtype == 1) return D == 64 ? launch<bf16_t, 64>(a, stream) : launch<bf16_t, 128>(a, stream);
    return D == 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace gdr
