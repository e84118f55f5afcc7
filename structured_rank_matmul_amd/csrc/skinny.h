// Streaming products for few tokens (skinny.hip, moe.hip): each wavefront runs
// its own stream of slabs from global memory through a ring in LDS, with no
// barrier, so that the loads of the slabs ahead are always in flight.
//
// A slab is 128 bytes of K of 16 weight rows (and, where they do not fit in
// registers, of 16 token rows), copied by buffer loads that write LDS: 8 rows of
// 128 bytes (whole cache lines) an instruction, no registers held.  Row r keeps
// chunk c (16 bytes) at position c ^ (r / 2 % 8), so the fragment reads are free
// of bank conflicts; a chunk past the end of K is read out of the buffer's
// range, which gives zeros.
//
// This pattern alone, without the tokens and the products, streams 235 MB of
// 8 KB rows in 38.4 us (6.1 TB/s); the best plain register stream of the same
// bytes takes 34.9 (6.7 TB/s).
#pragma once

#include "ffn_tile.h"

namespace dyra {

// This lane's part of the copies of 16 rows: row 8 q + lane / 8, q = 0, 1, and
// the chunk (byte offset) that the swizzle puts at its place.
__device__ __forceinline__ int slab_row(int q) { return 8 * q + ((threadIdx.x & 63) >> 3); }
__device__ __forceinline__ uint32_t slab_chunk(int q) {
    const int lane = threadIdx.x & 63;
    return 16u * (((lane & 7) ^ (lane >> 4)) ^ (4 * q));
}
// Where 16 rows lie: the buffer of rows 8 q .. and this lane's offset in it.
struct SlabRows {
    __amdgpu_buffer_rsrc_t buf[2];
    uint32_t off[2];
};

// Fragments of one slab: 128 bytes of K are STEPS steps of 32 elements.
template <typename E> struct SlabFrag {
    static constexpr int STEPS = 128 / (32 * (int)sizeof(E));
    typename Frag<E>::type f[STEPS];
};
__device__ __forceinline__ f32x4 slab_product(f32x4 acc, const SlabFrag<bf16> &w, const SlabFrag<bf16> &x) {
    return mma32(mma32(acc, w.f[0], x.f[0]), w.f[1], x.f[1]);
}
__device__ __forceinline__ f32x4 slab_product(f32x4 acc, const SlabFrag<float> &w, const SlabFrag<float> &x) {
    return mma32(acc, w.f[0], x.f[0]);
}
// The fragments of row `lane % ROWS` of a slab in LDS.
template <typename E, int ROWS> __device__ __forceinline__ SlabFrag<E> slab_read(const char *slab) {
    const int lane = threadIdx.x & 63, r16 = lane & (ROWS - 1), g = lane >> 4, sw = r16 >> 1;
    const char *p = slab + r16 * 128;
    SlabFrag<E> r;
    if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) r.f[h] = *reinterpret_cast<const bf16x8 *>(p + (((4 * h + g) ^ sw) << 4));
    } else {
        const f32x4 lo = *reinterpret_cast<const f32x4 *>(p + (((2 * g) ^ sw) << 4));
        const f32x4 hi = *reinterpret_cast<const f32x4 *>(p + (((2 * g + 1) ^ sw) << 4));
        r.f[0] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return r;
}
// The same fragments from global memory: `row` this lane's row offset in the
// buffer, `k` the slab's first byte, `left` the bytes of the rows from there on.
template <typename E> __device__ __forceinline__ SlabFrag<E> slab_load(__amdgpu_buffer_rsrc_t buf, uint32_t row, uint32_t k,
                                                                      int left) {
    const uint32_t g = (threadIdx.x & 63) >> 4;
    SlabFrag<E> r;
    auto chunk = [&](uint32_t c) -> u32x4 {
        // (a row at kOutside stays outside: zeros)
        return __builtin_amdgcn_raw_buffer_load_b128(buf, (int)(16 * c) < left ? row + 16 * c : kOutside, (int)k, 0);
    };
    if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) r.f[h] = __builtin_bit_cast(bf16x8, chunk(4 * h + g));
    } else {
        const f32x4 lo = __builtin_bit_cast(f32x4, chunk(2 * g)), hi = __builtin_bit_cast(f32x4, chunk(2 * g + 1));
        r.f[0] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return r;
}

constexpr int kRingBytes = 16384;  // of LDS for each wavefront's ring

// One wavefront's ring of slabs: of weights, or (TOKENS) of weights and tokens.
// WROWS: 16 weight rows a slab, or 8 (rows 8 .. 15 of the fragments repeat them).
template <typename E, bool TOKENS, int WROWS = 16> struct SlabRing {
    static constexpr int WBYTES = 128 * WROWS, SLAB = WBYTES + (TOKENS ? 2048 : 0);
    static constexpr int DEPTH = kRingBytes / SLAB, COPIES = WROWS / 8 + (TOKENS ? 2 : 0);
    char *ring;            // this wavefront's kRingBytes of LDS
    int ahead = 0;             // slabs issued and not consumed
    int put = 0, got = 0;      // places of the next slab to issue and to consume

    template <int ROWS> __device__ __forceinline__ void copy(const SlabRows &r, uint32_t k, int left, char *dst) {
#pragma unroll
        for (int q = 0; q < ROWS / 8; ++q)
            buffer_to_lds16(r.buf[q], (int)slab_chunk(q) < left ? r.off[q] : kOutside, k, dst + 1024 * q);
    }
    // Copies one slab at byte `k` of the rows; `left` bytes of the rows are left.
    __device__ __forceinline__ void issue(const SlabRows &w, const SlabRows &x, uint32_t k, int left) {
        char *dst = ring + put * SLAB;
        copy<WROWS>(w, k, left, dst);
        if constexpr (TOKENS) copy<16>(x, k, left, dst + WBYTES);
        put = put + 1 == DEPTH ? 0 : put + 1;
        ++ahead;
    }
    // Waits for the oldest slab and reads its fragments; its place is then free.
    __device__ __forceinline__ void take(SlabFrag<E> &w, SlabFrag<E> &x) {
        // (stores issued in between only make the wait stricter)
        if (ahead == DEPTH) wait_vmcnt<(DEPTH - 1) * COPIES>();
        else wait_vmcnt<0>();
        // the copies write LDS behind the compiler's back: no read may move above the wait
        asm volatile("" ::: "memory");
        const char *slab = ring + got * SLAB;
        w = slab_read<E, WROWS>(slab);
        if constexpr (TOKENS) x = slab_read<E, 16>(slab + WBYTES);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the fragments are in registers
        asm volatile("" ::: "memory");
        got = got + 1 == DEPTH ? 0 : got + 1;
        --ahead;
    }
};

}  // namespace dyra
