// MFMA operands of eight consecutive elements to a lane, and tiles of rows in LDS
// that give them along a row or down a column.
#pragma once

#include "gdn_device.hpp"

namespace gdn {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// Eight consecutive elements of the contraction in each lane, lane group g of
// 16 at 8g..8g+7 of 32: one MFMA for bf16, eight of four for fp32 (whose order
// inside the 32 differs, alike in both operands).
template <typename T> struct Eight;
template <> struct Eight<bf16> {
    typedef bf16x8 frag;
    static constexpr int PARTS = 3;
    __device__ __forceinline__ static frag pack(const float* f) { return __builtin_bit_cast(frag, Vec16<bf16>::pack(f)); }
    __device__ __forceinline__ static void unpack(frag a, float* f) {
        const u32x4 r = __builtin_bit_cast(u32x4, a);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(r[e] << 16);
            f[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
        }
    }
    // f as a sum of N parts: upper halves taken off one by one, the last part rounded (of three
    // parts, 24 bits, nothing is left to round).  Masks, subtractions and byte permutes run at two
    // to four times the rate of conversions.
    template <int N> __device__ __forceinline__ static void split(const float* f, frag* p) {
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = f[e];
#pragma unroll
        for (int i = 0; i + 1 < N; ++i) p[i] = take(r);
        p[N - 1] = N == 3 ? take(r) : pack(r);
    }
    // the upper halves of r, which keeps the rest
    __device__ __forceinline__ static frag take(float* r) {
        u32x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = __builtin_amdgcn_perm(__float_as_uint(r[2 * e + 1]), __float_as_uint(r[2 * e]), 0x07060302u);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] -= __uint_as_float(__float_as_uint(r[e]) & 0xffff0000u);
        return __builtin_bit_cast(frag, h);
    }
    __device__ __forceinline__ static f32x4 mma(frag a, frag b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Eight<float> {
    typedef f32x8 frag;
    static constexpr int PARTS = 1;
    __device__ __forceinline__ static frag pack(const float* f) {
        return frag{f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
    }
    __device__ __forceinline__ static void unpack(frag a, float* f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = a[e];
    }
    template <int N> __device__ __forceinline__ static void split(const float* f, frag* p) { p[0] = pack(f); }
    __device__ __forceinline__ static f32x4 mma(frag a, frag b, f32x4 c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
};

// Rows of D elements in LDS, 16 bytes apart beyond their width: rows of one column
// then start in different banks, and every address is one register and a constant.
// The gap of a row holds four floats for whoever wants them.
template <typename T, int D> struct Rows {
    static constexpr int U = 16 / sizeof(T), UR = D / U, PITCH = D + U;
    typedef typename Eight<T>::frag frag;
    T* p;
    __device__ __forceinline__ static int at(int row, int d) { return row * PITCH + d; }
    __device__ __forceinline__ float* gap(int row) const { return reinterpret_cast<float*>(p + at(row, D)); }
    // elements d .. d+7 of a row (d a multiple of 8)
    __device__ __forceinline__ frag row8(int row, int d) const {
        if constexpr (sizeof(T) == 2) {
            return *reinterpret_cast<const frag*>(p + at(row, d));
        } else {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(p + at(row, d));
            const f32x4 hi = *reinterpret_cast<const f32x4*>(p + at(row, d + 4));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // elements d .. d+3 and d+16 .. d+19 of a row (d a multiple of 4): the order in which an
    // accumulator's two tiles of 16 rows hold theirs
    __device__ __forceinline__ frag row44(int row, int d) const {
        if constexpr (sizeof(T) == 2) {
            const u32x2 lo = *reinterpret_cast<const u32x2*>(p + at(row, d));
            const u32x2 hi = *reinterpret_cast<const u32x2*>(p + at(row, d + 16));
            return __builtin_bit_cast(frag, u32x4{lo.x, lo.y, hi.x, hi.y});
        } else {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(p + at(row, d));
            const f32x4 hi = *reinterpret_cast<const f32x4*>(p + at(row, d + 16));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // elements d .. d+3 of a row in fp32 (d a multiple of 4)
    __device__ __forceinline__ f32x4 row4(int row, int d) const {
        return Quad<T>::get(Quad<T>::load(p + at(row, d)));
    }
    // Transposed: lane r of a group of 16 gets column d0 + 8 (r / 4) + r % 4 (d0 a multiple of
    // 4; SPREAD false: d0 + r) at rows t0 + 4g + 0..3 and t0 + 16 + 4g + 0..3.
    template <bool SPREAD> __device__ __forceinline__ frag col8(int t0, int d0, int lane) const {
        const int g = lane >> 4, r = lane & 15;
        if constexpr (sizeof(T) == 2) {
            // lane j of the group addresses row (j / 4), four columns at j % 4 (see Mma::load_t)
            const int row = t0 + 4 * g + (r >> 2), d = d0 + (SPREAD ? 8 : 4) * (r & 3);
            typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
            typedef short i16x8 __attribute__((ext_vector_type(8)));
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + at(row, d)));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + at(row + 16, d)));
            return __builtin_bit_cast(frag, (i16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int d = d0 + (SPREAD ? 8 * (r >> 2) + (r & 3) : r);
            frag v;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = t0 + 4 * g + (e & 3) + 4 * (e & 4);
                v[e] = p[at(row, d)];
            }
            return v;
        }
    }
    // The same with 16 rows: rows 4g + 0..3, and zeros.
    __device__ __forceinline__ frag col4(int d0, int lane) const {
        const int g = lane >> 4, r = lane & 15;
        if constexpr (sizeof(T) == 2) {
            typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + at(4 * g + (r >> 2), d0 + 4 * (r & 3))));
            const u32x2 x = __builtin_bit_cast(u32x2, lo);
            return __builtin_bit_cast(frag, u32x4{x.x, x.y, 0, 0});
        } else {
            frag v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < 4 ? p[at(4 * g + e, d0 + r)] : 0.f;
            return v;
        }
    }
};

}  // namespace gdn
