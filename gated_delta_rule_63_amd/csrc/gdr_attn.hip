// Causal attention over packed prompts (gdr_attn_prefill_fwd).
//
// A workgroup owns 128 consecutive tokens of the packed batch and one query head: four waves of 32 query rows.
// Tiles of 64 keys and values go through the LDS once for all four.  The tokens are cut at fixed borders, not at
// those of the sequences: a tile may hold several sequences' rows, each row sees the tokens from its sequence's
// start to itself, and 128 one-token sequences are one workgroup's work.
#include <hip/hip_runtime.h>

#include "gdr_attn_device.h"

namespace gdr {
namespace {

constexpr int kRows = 128, kKeys = 64;

template <typename T, int D>
__global__ __launch_bounds__(256, 2) void attn_prefill_kernel(AttnPrefillArgs a) {
    using L = AttnTile<T, D>;
    using C = AttnCore<T, D>;
    __shared__ __align__(1024) char lds[2 * kKeys * L::row_bytes];
    char* const sk = lds;
    char* const sv = lds + kKeys * L::row_bytes;

    int tile, head;
    {
        const int b = blockIdx.x;
        if (a.HQ % 8 == 0) {  // workgroups go round the eight XCDs: each keeps to its own heads' keys and values
            const int per = a.HQ / 8, x = b & 7, i = b >> 3;
            tile = a.tiles - 1 - i / per;
            head = x * per + i % per;
        } else {
            tile = a.tiles - 1 - b / a.HQ;
            head = b % a.HQ;
        }
    }
    const int end = a.cu ? a.cu[a.N] : (int)a.T;
    const int t0 = tile * kRows;
    if (t0 >= end) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
    const int kvh = head / (a.HQ / a.HK);
    const int t = t0 + 32 * wave + (lane & 31);
    const int tc = min(t, end - 1);
    const int start = a.cu ? a.cu[find_seq(a.cu, a.N, tc)] : 0;
    const int lo = a.cu ? a.cu[find_seq(a.cu, a.N, t0)] : 0;
    const int wlo = __builtin_amdgcn_readfirstlane(start), wfirst = t0 + 32 * wave;
    const int wlate = __builtin_amdgcn_readlane(start, 31);
    const int hi = min(t0 + kRows, end), whi = min(wfirst + 32, end);

    typename C::Q q;
    C::load_q(static_cast<const char*>(a.q) + ((int64_t)tc * a.q_stride + (int64_t)head * D) * L::es, half, a.negate, q);
    f32x16_t o[D / 32] = {};
    float m = kNegInf, l = 0.0f;
    const char* const kb = static_cast<const char*>(a.k) + (int64_t)kvh * D * L::es;
    const char* const vb = static_cast<const char*>(a.v) + (int64_t)kvh * D * L::es;

    for (int j0 = lo; j0 < hi; j0 += kKeys) {
        L::template stage<kKeys, 4, false>(sk, wave, lane, [&](int r) { return kb + (int64_t)min(j0 + r, end - 1) * a.k_stride * L::es; });
        L::template stage<kKeys, 4, true>(sv, wave, lane, [&](int r) { return vb + (int64_t)min(j0 + r, end - 1) * a.v_stride * L::es; });
        wait_loads();
        __syncthreads();
        if (j0 < whi && j0 + kKeys > wlo) {
            f32x16_t s[2] = {C::scores(sk, 0, lane, q), C::scores(sk, 1, lane, q)};
            if (j0 + kKeys - 1 > wfirst || j0 < wlate) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = j0 + 32 * b + key_of(i, half);
                        s[b][i] = j >= start && j <= t ? s[b][i] : kNegInf;
                    }
            }
            float mx = s[0][0];
#pragma unroll
            for (int i = 0; i < 32; ++i) mx = fmaxf(mx, s[i >> 4][i & 15]);
            const float mn = fmaxf(m, both_max(mx));
            const float base = mn == kNegInf ? 0.0f : mn * a.c;
            const float alpha = __builtin_amdgcn_exp2f(m * a.c - base);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int b = 0; b < D / 32; ++b) o[b] *= alpha;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[i >> 4][i & 15], a.c, -base));
                s[i >> 4][i & 15] = p;
                l += p;
            }
            C::accumulate(sv, 0, lane, s[0], o);
            C::accumulate(sv, 1, lane, s[1], o);
        }
        __syncthreads();
    }
    l = both_sum(l);
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
    char* row = t < end ? static_cast<char*>(a.o) + ((int64_t)t * a.HQ + head) * L::row_bytes : nullptr;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
        o[b] *= inv;
        C::store(row, b, half, o[b]);
    }
    if (a.lse && t < end && half == 0)
        a.lse[(int64_t)t * a.HQ + head] = l == 0.0f ? kNegInf : (m * a.c + __builtin_amdgcn_logf(l)) * kLn2;
}

template <typename T, int D>
hipError_t launch(const AttnPrefillArgs& a, hipStream_t stream) {
    attn_prefill_kernel<T, D><<<dim3((unsigned)(a.tiles * a.HQ)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t attn_prefill_tiles(int64_t T) { return (T + kRows - 1) / kRows; }

hipError_t launch_attn_prefill(AttnPrefillArgs a, int D, int io_dtype, hipStream_t stream) {
    a.tiles = (int)attn_prefill_tiles(a.T);
    if (io_dtype == 1) return D == 64 ? launch<bf16_t, 64>(a, stream) : launch<bf16_t, 128>(a, stream);
    return D == 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace gdr
