// Device code shared by the attention kernels: tiles of keys and values staged in the LDS, score tiles, the
// running softmax and the products with the values, on 32 x 32 matrix tiles.
//
// Everything is held transposed: S^T = K Q^T and O^T = V^T P^T.  In the matrix instructions' output layout a lane
// then holds values of one query row (column l % 32) only, so that the row's maximum, sum and rescaling factor
// are one register each and need one exchange, between a lane and its partner 32 away.  The score registers are
// at the same time the second product's B operand: its contraction index runs over the keys in the order in
// which the lanes hold them, and V^T is read in that order.
#pragma once

#include "gdr_device.h"
#include "gdr_internal.h"

namespace gdr {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

// value of the partner lane l ^ 32
__device__ __forceinline__ float other_half(float x) {
    const unsigned u = __float_as_uint(x);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);  // [lower half twice, upper half twice]
    return __uint_as_float((threadIdx.x & 32) ? p[0] : p[1]);
}
__device__ __forceinline__ float both_max(float x) {
    const unsigned u = __float_as_uint(x);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float both_sum(float x) {
    const unsigned u = __float_as_uint(x);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// 16 bytes per lane from global memory to lds + 16 * lane (lds is the wave's)
__device__ __forceinline__ void copy_to_lds(const char* g, char* lds) {
    __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) const void*)(g),
                                     (__attribute__((address_space(3))) void*)(lds), 16, 0, 0);
}

// sequence of a token below cu[N]: the last n with cu[n] <= t (so an empty sequence is never found)
__device__ __forceinline__ int find_seq(const int32_t* cu, int N, int t) {
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Layout of a staged tile: rows of D elements in 16-byte chunks, chunk c of row r at place c ^ swizzle(r), so that
// neither the score product's reads (the same chunk of consecutive rows) nor the transposing reads of V (four
// rows, two chunks each) meet in a bank.  The copy to the LDS writes 64 consecutive places per instruction;
// the lanes fetch the chunks that belong there.
template <typename T, int D> struct AttnTile {
    static constexpr int es = Elem<T>::bytes;
    static constexpr int row_bytes = D * es;
    static constexpr int chunks = row_bytes / 16;
    __device__ __forceinline__ static int swz_k(int row) { return row & 7; }
    __device__ __forceinline__ static int swz_v(int row) { return es == 2 ? (row & 3) << 1 : 0; }

    // rows [0, ROWS) of a tile by WAVES waves; at(row) gives a row's address
    template <int ROWS, int WAVES, bool V, typename F>
    __device__ __forceinline__ static void stage(char* lds, int wave, int lane, F at) {
        constexpr int per = ROWS * chunks / 64 / WAVES;
        static_assert(per * 64 * WAVES == ROWS * chunks, "whole instructions");
#pragma unroll
        for (int i = 0; i < per; ++i) {
            const int first = (wave * per + i) * 64;
            const int place = first + lane;
            const int row = place / chunks;
            const int c = (place % chunks) ^ (V ? swz_v(row) : swz_k(row));
            copy_to_lds(at(row) + 16 * c, lds + 16 * first);
        }
    }
};

// ---- products on 32 query rows, 32 keys at a time ---------------------------------------------------------
// Lane l: query row l % 32, half l / 32.  Score register i of a block is key 8 (i / 4) + 4 half + i % 4.
__device__ __forceinline__ int key_of(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

template <typename T, int D> struct AttnCore;

template <int D> struct AttnCore<bf16_t, D> {
    using L = AttnTile<bf16_t, D>;
    static constexpr int steps = D / 16;
    typedef bf16x8_t Q[steps];
    // chunk 2 s + half of the lane's query row
    __device__ __forceinline__ static void load_q(const char* row, int half, bool negate, Q& q) {
        const uint32_t flip = negate ? 0x80008000u : 0u;
#pragma unroll
        for (int s = 0; s < steps; ++s) {
            uint4 w = *reinterpret_cast<const uint4*>(row + 16 * (2 * s + half));
            w.x ^= flip; w.y ^= flip; w.z ^= flip; w.w ^= flip;
            q[s] = __builtin_bit_cast(bf16x8_t, w);
        }
    }
    __device__ __forceinline__ static f32x16_t scores(const char* k, int block, int lane, const Q& q) {
        const int row = 32 * block + (lane & 31), half = lane >> 5;
        f32x16_t acc = {};
#pragma unroll
        for (int s = 0; s < steps; ++s) {
            const bf16x8_t a = *reinterpret_cast<const bf16x8_t*>(k + row * L::row_bytes + 16 * ((2 * s + half) ^ L::swz_k(row)));
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[s], acc, 0, 0, 0);
        }
        return acc;
    }
    // V^T operand: channels 32 b + l % 32, the 16 keys of half-block t of a block, in the scores' order
    __device__ __forceinline__ static bf16x8_t values(const char* v, int block, int t, int b, int lane) {
        typedef short v4i16 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
        const int grp = lane >> 4, r = (lane >> 2) & 3;
        const int row = 32 * block + 16 * t + 4 * (grp >> 1) + r;
        const int c = 4 * b + 2 * (grp & 1) + ((lane & 3) >> 1);
        const char* p = v + row * L::row_bytes + 16 * (c ^ L::swz_v(r)) + 8 * (lane & 1);
        const v4i16 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p));
        const v4i16 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 8 * L::row_bytes));
        return __builtin_bit_cast(bf16x8_t, s16x8_t{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
    }
    __device__ __forceinline__ static void accumulate(const char* v, int block, int lane, const f32x16_t& p, f32x16_t* o) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint4 w;
            w.x = pack_bf16x2(p[8 * t + 0], p[8 * t + 1]);
            w.y = pack_bf16x2(p[8 * t + 2], p[8 * t + 3]);
            w.z = pack_bf16x2(p[8 * t + 4], p[8 * t + 5]);
            w.w = pack_bf16x2(p[8 * t + 6], p[8 * t + 7]);
            const bf16x8_t pb = __builtin_bit_cast(bf16x8_t, w);
#pragma unroll
            for (int b = 0; b < D / 32; ++b)
                o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(values(v, block, t, b, lane), pb, o[b], 0, 0, 0);
        }
    }
    // the lane's 16 values of channels 32 b .. 32 b + 31 (after the exchange 16 half .. + 15 in two runs of eight)
    __device__ __forceinline__ static void store(char* row, int b, int half, const f32x16_t& o) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t a0 = pack_bf16x2(o[8 * g + 0], o[8 * g + 1]), a1 = pack_bf16x2(o[8 * g + 2], o[8 * g + 3]);
            uint32_t b0 = pack_bf16x2(o[8 * g + 4], o[8 * g + 5]), b1 = pack_bf16x2(o[8 * g + 6], o[8 * g + 7]);
            const auto x = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
            if (row) *reinterpret_cast<uint4*>(row + 64 * b + 32 * g + 16 * half) = uint4{x[0], y[0], x[1], y[1]};
        }
    }
};

template <int D> struct AttnCore<float, D> {
    using L = AttnTile<float, D>;
    static constexpr int steps = D / 8;
    typedef f32x4_t Q[steps];
    __device__ __forceinline__ static void load_q(const char* row, int half, bool negate, Q& q) {
        const float sign = negate ? -1.0f : 1.0f;
#pragma unroll
        for (int s = 0; s < steps; ++s) q[s] = *reinterpret_cast<const f32x4_t*>(row + 16 * (2 * s + half)) * sign;
    }
    __device__ __forceinline__ static f32x16_t scores(const char* k, int block, int lane, const Q& q) {
        const int row = 32 * block + (lane & 31), half = lane >> 5;
        f32x16_t acc = {};
#pragma unroll
        for (int s = 0; s < steps; ++s) {
            const f32x4_t a = *reinterpret_cast<const f32x4_t*>(k + row * L::row_bytes + 16 * ((2 * s + half) ^ L::swz_k(row)));
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], q[s][e], acc, 0, 0, 0);
        }
        return acc;
    }
    __device__ __forceinline__ static float value(const char* v, int block, int i, int b, int lane) {
        const int row = 32 * block + key_of(i, lane >> 5);
        return *reinterpret_cast<const float*>(v + row * L::row_bytes + 4 * (32 * b + (lane & 31)));
    }
    __device__ __forceinline__ static void accumulate(const char* v, int block, int lane, const f32x16_t& p, f32x16_t* o) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int b = 0; b < D / 32; ++b)
                o[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(value(v, block, i, b, lane), p[i], o[b], 0, 0, 0);
    }
    __device__ __forceinline__ static void store(char* row, int b, int half, const f32x16_t& o) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (row)
                *reinterpret_cast<f32x4_t*>(row + 128 * b + 32 * g + 16 * half) =
                    f32x4_t{o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]};
    }
};

}  // namespace gdr
