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

// ---- asynchronous copies to the LDS -------------------------------------------------------------------------
// 16 bytes per lane from base + off to lds + 16 * lane (base and lds are the wave's).  Written as assembly because
// the compiler, which cannot tell a tile being filled from the one being read, would otherwise wait for the copies
// in flight before the first transposing read; nothing is returned in registers, and wait_copies() is the wait
// that the copies need before a barrier makes them visible.
typedef __attribute__((address_space(3))) const char lds_char;
__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(uintptr_t)(lds_char*)(p); }
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32 | (uint32_t)uniform((int)x));
}
// A base address for copies: in scalar registers, and settled there, should a vector instruction have written them
// (five wait states, of which the copy has two; the compiler does not look into assembly for this).
__device__ __forceinline__ const char* copy_base(const char* p) {
    p = reinterpret_cast<const char*>(uniform((int64_t)reinterpret_cast<uintptr_t>(p)));
    asm volatile("s_nop 3" : "+s"(p));
    return p;
}
__device__ __forceinline__ void copy_to_lds(const char* base, uint32_t off, uint32_t lds) {
    lds = (uint32_t)uniform((int)lds);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 : : "v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
// until at most LEFT of the wave's copies, the last ones, are on their way
template <int LEFT = 0> __device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(%0)" : : "n"(LEFT) : "memory"); }

// inclusive sum over the lanes of a wave
template <int CTRL, int ROWS, bool ZERO> __device__ __forceinline__ int dpp_add(int x) {
    return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, ZERO);
}
__device__ __forceinline__ int wave_scan(int x) {
    x = dpp_add<0x111, 0xF, true>(x);    // row_shr 1, 2, 4, 8: within rows of 16 lanes
    x = dpp_add<0x112, 0xF, true>(x);
    x = dpp_add<0x114, 0xF, true>(x);
    x = dpp_add<0x118, 0xF, true>(x);
    x = dpp_add<0x142, 0xA, false>(x);   // row 0's total to row 1, row 2's to row 3
    x = dpp_add<0x143, 0xC, false>(x);   // that of rows 0 and 1 to rows 2 and 3
    return x;
}
__device__ __forceinline__ int lane_value(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ int wave_max(int x) {   // x >= 0
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));
    return lane_value(x, 63);
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
// rows, two chunks each) meet in a bank.  A copy writes 64 consecutive places per instruction; the lanes fetch
// the chunks that belong there.
template <typename T, int D> struct AttnTile {
    static constexpr int es = Elem<T>::bytes;
    static constexpr int row_bytes = D * es;
    static constexpr int chunks = row_bytes / 16;
    // so many rows' reads of one chunk meet all places of 256 bytes
    __device__ __forceinline__ static int swz_k(int row) { return chunks >= 16 ? row & 15 : (row >> 1) & 7; }
    // step s of a lane's reads of a key row (chunk 2 s + half) is at register s % regs, 32 regs bytes on for each turn
    static constexpr int regs = chunks >= 16 ? 8 : 4;
    __device__ __forceinline__ static int swz_v(int row) { return es == 2 ? (row & 3) << (chunks >= 16 ? 2 : 1) : 0; }
    // instruction i of a wave's copies fills the places 64 (per * wave + i) ..; the lane's row and byte in the row
    template <int ROWS, int WAVES> static constexpr int per() { return ROWS * chunks / 64 / WAVES; }
    __device__ __forceinline__ static int copy_row(int first, int lane) { return (first + lane) / chunks; }
    template <bool V> __device__ __forceinline__ static int copy_byte(int first, int lane) {
        const int row = copy_row(first, lane);
        return 16 * (((first + lane) % chunks) ^ (V ? swz_v(row) : swz_k(row)));
    }
};

// what is behind is not begun before
__device__ __forceinline__ void apart() { asm volatile("" ::: "memory"); }
__device__ __forceinline__ void hide_int(uint32_t& x) { asm volatile("" : "+v"(x)); }

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
    // Addresses of the lane's reads in a tile: the rest is in the instructions' offsets
    struct At {
        uint32_t k[L::regs], v[D / 32];
        __device__ __forceinline__ void move(uint32_t by) {
#pragma unroll
            for (int s = 0; s < L::regs; ++s) hide_int(k[s] += by);
#pragma unroll
            for (int b = 0; b < D / 32; ++b) hide_int(v[b] += by);
        }
        __device__ __forceinline__ At(uint32_t k0, uint32_t v0, int lane) {
            const int row = lane & 31, half = lane >> 5, grp = lane >> 4, r = (lane >> 2) & 3;
#pragma unroll
            for (int s = 0; s < L::regs; ++s) k[s] = k0 + row * L::row_bytes + 16 * ((2 * s + half) ^ L::swz_k(row));
#pragma unroll
            for (int b = 0; b < D / 32; ++b)
                v[b] = v0 + (4 * (grp >> 1) + r) * L::row_bytes + 16 * ((4 * b + 2 * (grp & 1) + ((lane & 3) >> 1)) ^ L::swz_v(r)) +
                       8 * (lane & 1);
        }
    };
    __device__ __forceinline__ static f32x16_t scores(int block, const At& at, const Q& q) {
        typedef __attribute__((address_space(3))) const bf16x8_t lds_v8;
        f32x16_t acc = {};
#pragma unroll
        for (int s = 0; s < steps; ++s) {
            const bf16x8_t a = *(lds_v8*)(uintptr_t)(at.k[s % L::regs] + (32 * L::regs * (s / L::regs) + 32 * block * L::row_bytes));
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[s], acc, 0, 0, 0);
        }
        return acc;
    }
    // V^T operand: channels 32 b + l % 32, the 16 keys of half-block t of a block, in the scores' order
    __device__ __forceinline__ static bf16x8_t values(int block, int t, int b, const At& at) {
        typedef short v4i16 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
        const uint32_t off = (32 * block + 16 * t) * L::row_bytes;
        const v4i16 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)(at.v[b] + off));
        const v4i16 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)(at.v[b] + (off + 8 * L::row_bytes)));
        return __builtin_bit_cast(bf16x8_t, s16x8_t{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
    }
    // o += V^T p, with the weights rounded to bf16, which the matrix instruction takes: a second product with what the rounding
    // leaves would be half of all products once more.  The weights are relative to the running reference, so each is off by up
    // to 2^-8 of itself; their sum takes them as they are, for the sake of lse.  Outputs of 8 ragged prompts of 32768 tokens
    // together are off by 0.0022 of their size (0.0016 of it is the rounding of o).
    __device__ __forceinline__ static void accumulate(int block, const At& at, const f32x16_t& p, f32x16_t* o, float& l) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = pack_bf16x2(p[8 * t + 2 * i], p[8 * t + 2 * i + 1]);
                l += p[8 * t + 2 * i] + p[8 * t + 2 * i + 1];
            }
            const bf16x8_t pb = __builtin_bit_cast(bf16x8_t, uint4{w[0], w[1], w[2], w[3]});
#pragma unroll
            for (int b = 0; b < D / 32; ++b)
                o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(values(block, t, b, at), pb, o[b], 0, 0, 0);
        }
    }
    // elements of a 32-bit word that are not finite: all bits of theirs
    __device__ __forceinline__ static uint32_t not_finite(uint32_t w) {
        const uint32_t m = ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
        return m | (m - (m >> 15));
    }
    // o += the values of a row in global memory that are not finite
    __device__ __forceinline__ static void add_specials(const char* row, int half, f32x16_t* o) {
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint2 w = *reinterpret_cast<const uint2*>(row + 64 * b + 16 * g + 8 * half);
                const uint32_t x[4] = {w.x << 16, w.x & 0xFFFF0000u, w.y << 16, w.y & 0xFFFF0000u};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f = __uint_as_float(x[e]);
                    o[b][4 * g + e] += __builtin_isfinite(f) ? 0.0f : f;
                }
                apart();
            }
    }
    // the lane's half of its query row; the halves exchange values so that each writes runs of eight
    __device__ __forceinline__ static void store(char* row, int half, const f32x16_t* o) {
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t a0 = pack_bf16x2(o[b][8 * g + 0], o[b][8 * g + 1]), a1 = pack_bf16x2(o[b][8 * g + 2], o[b][8 * g + 3]);
                const uint32_t b0 = pack_bf16x2(o[b][8 * g + 4], o[b][8 * g + 5]), b1 = pack_bf16x2(o[b][8 * g + 6], o[b][8 * g + 7]);
                const auto x = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
                const auto y = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
                if (row) *reinterpret_cast<uint4*>(row + 64 * b + 32 * g + 16 * half) = uint4{x[0], y[0], x[1], y[1]};
            }
    }
    __device__ __forceinline__ static void store_part(float* row, int half, const f32x16_t* o) {
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4_t*>(row + 32 * b + 8 * g + 4 * half) =
                    f32x4_t{o[b][4 * g], o[b][4 * g + 1], o[b][4 * g + 2], o[b][4 * g + 3]};
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
    // Row r of channel block b stands for channel (D / 32) r + b, so that a lane's operands of all blocks are
    // neighbours.
    static constexpr int nb = D / 32;
    typedef float vec_t __attribute__((ext_vector_type(nb)));
    struct At {
        uint32_t k[L::regs], v;
        __device__ __forceinline__ void move(uint32_t by) {
#pragma unroll
            for (int s = 0; s < L::regs; ++s) hide_int(k[s] += by);
            hide_int(v += by);
        }
        __device__ __forceinline__ At(uint32_t k0, uint32_t v0, int lane) {
            const int row = lane & 31, half = lane >> 5;
#pragma unroll
            for (int s = 0; s < L::regs; ++s) k[s] = k0 + row * L::row_bytes + 16 * ((2 * s + half) ^ L::swz_k(row));
            v = v0 + 4 * half * L::row_bytes + 4 * nb * row;
        }
    };
    __device__ __forceinline__ static f32x16_t scores(int block, const At& at, const Q& q) {
        typedef __attribute__((address_space(3))) const f32x4_t lds_v4;
        f32x16_t acc = {};
#pragma unroll
        for (int s = 0; s < steps; ++s) {
            const f32x4_t a = *(lds_v4*)(uintptr_t)(at.k[s % L::regs] + (32 * L::regs * (s / L::regs) + 32 * block * L::row_bytes));
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], q[s][e], acc, 0, 0, 0);
        }
        return acc;
    }
    __device__ __forceinline__ static void accumulate(int block, const At& at, const f32x16_t& p, f32x16_t* o, float& l) {
        typedef __attribute__((address_space(3))) const vec_t lds_vec;
        vec_t a[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = *(lds_vec*)(uintptr_t)(at.v + (32 * block + key_of(i, 0)) * L::row_bytes);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            l += p[i];
#pragma unroll
            for (int b = 0; b < nb; ++b) o[b] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i][b], p[i], o[b], 0, 0, 0);
        }
    }
    __device__ __forceinline__ static uint32_t not_finite(uint32_t w) { return (w & 0x7F800000u) == 0x7F800000u ? ~0u : 0u; }
    __device__ __forceinline__ static void add_specials(const char* row, int half, f32x16_t* o) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const vec_t x = *reinterpret_cast<const vec_t*>(row + 4 * nb * key_of(i, half));
#pragma unroll
            for (int b = 0; b < nb; ++b) o[b][i] += __builtin_isfinite(x[b]) ? 0.0f : x[b];
            apart();
        }
    }
    __device__ __forceinline__ static void store(char* row, int half, const f32x16_t* o) {
        if (row) store_part(reinterpret_cast<float*>(row), half, o);
    }
    __device__ __forceinline__ static void store_part(float* row, int half, const f32x16_t* o) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            vec_t x;
#pragma unroll
            for (int b = 0; b < nb; ++b) x[b] = o[b][i];
            *reinterpret_cast<vec_t*>(row + nb * key_of(i, half)) = x;
        }
    }
};

// ---- running softmax of a wave's 32 rows ----------------------------------------------------------------------
// Weights are e^(x - m) with x = scale * score and m a running reference: the maximum of the row so far, moved only
// when a score passes it by more than 2^8 (in which case what is there is rescaled).  The weights stay below 2^8,
// their sum far from fp32's range, and most tiles leave the output's registers alone.
constexpr float kSlack = 8.0f;

template <typename T, int D> struct AttnRow {
    using C = AttnCore<T, D>;
    f32x16_t o[D / 32] = {};
    float m = kNegInf;   // of the raw scores
    float l = 0.0f;      // sum of the lane's weights (its half of the keys)

    // adds NB blocks of scores; first: the first of these blocks in the tile
    template <int NB>
    __device__ __forceinline__ void add(f32x16_t (&s)[NB], float c, int first, const typename C::At& at) {
        float mx = s[0][0];
#pragma unroll
        for (int i = 1; i < 16 * NB; ++i) mx = fmaxf(mx, s[i >> 4][i & 15]);
        mx = both_max(mx);
        if (__any((mx - m) * c > kSlack || (m == kNegInf && mx > kNegInf))) {
            const float mn = fmaxf(m, mx);
            const float alpha = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((m - mn) * c);
            m = mn;
            l *= alpha;
#pragma unroll
            for (int b = 0; b < D / 32; ++b) o[b] *= alpha;
        }
        float base = m == kNegInf ? 0.0f : m * c;
        // Rounding m c moves all weights of the row by one factor of up to 2^(2^-24 m c).  Where that could leave fp32, or m c
        // itself does, the scores are taken relative to m before the scale.
        if (__any(__builtin_fabsf(base) > 0x1p24f)) {
            const float m0 = m == kNegInf ? 0.0f : m;
#pragma unroll
            for (int i = 0; i < 16 * NB; ++i) s[i >> 4][i & 15] -= m0;
            base = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 16 * NB; ++i) s[i >> 4][i & 15] = __builtin_amdgcn_exp2f(fmaf(s[i >> 4][i & 15], c, -base));
#pragma unroll
        for (int b = 0; b < NB; ++b) C::accumulate(first + b, at, s[b], o, l);
    }
};

// The parts of the KW waves with the same rows and different keys, joined in that with kw == 0: the upper half of the
// waves hands its parts to the lower half until one is left.  All waves of the workgroup call it.  place: KW / 2 times
// 64 lanes' outputs, stats: as many times two floats a lane, of the waves with the same rows.
template <int D, int KW>
__device__ __forceinline__ void join_waves(f32x16_t* o, float& m, float& l, float c, float* place, float* stats, int kw, int lane) {
#pragma unroll
    for (int n = KW / 2; n > 0; n /= 2) {
        float* const mine = place + (kw % n) * (64 * D / 2) + lane;
        float* const st = stats + (kw % n) * 128 + lane;
        __syncthreads();
        if (kw >= n && kw < 2 * n) {
            st[0] = m;
            st[64] = l;
#pragma unroll
            for (int b = 0; b < D / 32; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) mine[(16 * b + i) * 64] = o[b][i];
        }
        __syncthreads();
        if (kw < n) {
            const float m1 = st[0], l1 = st[64], mn = fmaxf(m, m1);
            const float e0 = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((m - mn) * c);
            const float e1 = m1 == kNegInf ? 0.0f : __builtin_amdgcn_exp2f((m1 - mn) * c);
#pragma unroll
            for (int b = 0; b < D / 32; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[b][i] = o[b][i] * e0 + mine[(16 * b + i) * 64] * e1;
            l = l * e0 + l1 * e1;
            m = mn;
        }
    }
}

// Values that are not finite, in a tile of which some row does not see some key: 0 * inf must not reach that row.
// Before the tile is used they become 0 in the LDS; the rows that see them then add them as they are.  rows[turn] holds
// a bit per key, in two turns: the other one is cleared here, behind the barrier that ends its use.
template <typename T, int D, int KEYS, int WAVES>
__device__ __forceinline__ void take_out_specials(uint32_t v, uint32_t (*rows)[KEYS / 32], int turn, int wave, int lane) {
    using L = AttnTile<T, D>;
    typedef __attribute__((address_space(3))) uint4 lds_u4;
    constexpr int per = L::template per<KEYS, WAVES>();
#pragma unroll
    for (int i = 0; i < per; ++i) {
        const int first = 64 * (per * wave + i);
        lds_u4* const p = (lds_u4*)(uintptr_t)(v + 16 * (first + lane));
        uint4 w{p->x, p->y, p->z, p->w};
        const uint4 bad{AttnCore<T, D>::not_finite(w.x), AttnCore<T, D>::not_finite(w.y), AttnCore<T, D>::not_finite(w.z),
                        AttnCore<T, D>::not_finite(w.w)};
        if (bad.x | bad.y | bad.z | bad.w) {
            const int row = L::copy_row(first, lane);
            atomicOr(&rows[turn][row >> 5], 1u << (row & 31));
            p->x = w.x & ~bad.x; p->y = w.y & ~bad.y; p->z = w.z & ~bad.z; p->w = w.w & ~bad.w;
        }
    }
    __syncthreads();
    if (threadIdx.x < KEYS / 32) rows[turn ^ 1][threadIdx.x] = 0;
}

// Weights without a sum: those of a row that saw nothing, whose output is 0 and lse -inf, or of one that saw scores of -inf
// only, whose softmax is 0 / 0.  The caller knows which, and says so by a sum that is a NaN.
__device__ __forceinline__ float no_sum() { return __builtin_nanf(""); }
// 1 / l; 0 for a row that saw nothing; a NaN stays one
__device__ __forceinline__ float reciprocal_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float log_sum(float base, float l) {
    return l == 0.0f ? kNegInf : (base + __builtin_amdgcn_logf(l)) * kLn2;
}

}  // namespace gdr
