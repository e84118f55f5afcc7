// Router and expert layer for a few tokens.
//
// Router: 16 or 64 lanes per row of logits, its values in registers; k rounds of
// an argmax over keys that order by (value, lower index first).  Bound by the
// rounds' lane exchanges: 8 of 128 logits in 16384 rows take 8.3 us (8.5 MB read), 8
// of 64 in 16 rows 3.1, little more than an empty kernel.
//
// Expert layer, two kernels (three where c is narrow).  moe_up forms H[pair][f] =
// act(X Wg_e^T) * (X Wu_e^T) for every (token, place) pair; moe_down forms Y = R +
// sum_j w_j H_j Wd_e^T.  Both are bound by reading the weights of the chosen experts
// once: a workgroup gathers the tokens of an expert and multiplies them together,
// the weights streamed through per-wavefront rings (skinny.h).  Every workgroup
// sorts the places by expert itself (a few LDS steps), so that two launches do.  No
// atomics on results: every pair's products have a place of their own in LDS and
// are added per token in the order of its places.  Up and down take 137 and 77 us
// for 48 tokens with 6 places over 64 experts of 2048 x 1408 (1.08 GB, 5.0 TB/s),
// 326 and 170 for 16 tokens with 2 over 8 of 4096 x 14336 (2.8 GB, 5.7 TB/s), 18.0
// and 10.7 for 1 token with 8 over 64 of 2048 x 1024 (101 MB, start-up included);
// float32, 48 tokens with 6 over 64 of 2048 x 704 (1.1 GB) 135 and 80.
//
// H between the two is a bf16 operand of the second product.  Rounded to it once,
// it alone puts 1e-3 of a result's size into every result, where the last rounding
// puts 1.66e-3 (error against float64, 16 tokens with 2 places over 8 experts of
// 4096 x 14336: 2.00e-3 against 1.66e-3).  So H keeps what the rounding left out as
// a second bf16 (together to 2^-16 of it), and the second product is taken of both
// parts: twice the ring bytes of the pairs, 10, 4 and 0.5 us of a call in the cases
// above, 34 of 192 at 512 tokens with 2 places over 8 experts of 1024 x 2816.  A caller whose
// workspace has no room for the second part has H rounded once.
#include "lanes.h"
#include "skinny.h"

#include <algorithm>

namespace dyra {

namespace {

// ------------------------------------------------------------------ router

// Orders like the float (-0 as +0), above 0 for every value that may be chosen.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// v of the lane whose number differs in bit D of a group of LANES (16: by DPP,
// inside a row of the wavefront; 64: across rows by LDS permute).
template <int D> __device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
    if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(v, 0xb1, 0xf, 0xf, true);        // quad_perm 1 0 3 2
    else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(v, 0x4e, 0xf, 0xf, true);   // quad_perm 2 3 0 1
    else if constexpr (D == 4) return __shfl_xor(v, 4);
    else if constexpr (D == 8) return __builtin_amdgcn_mov_dpp(v, 0x128, 0xf, 0xf, true);  // row_ror 8
    else return __shfl_xor(v, D);
}
template <int LANES, class F> __device__ __forceinline__ void butterfly(F &&f) {
    f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 4>{});
    f(std::integral_constant<int, 8>{});
    if constexpr (LANES == 64) {
        f(std::integral_constant<int, 16>{});
        f(std::integral_constant<int, 32>{});
    }
}
template <int LANES> __device__ __forceinline__ float lane_sum(float v) {
    butterfly<LANES>([&](auto d) __attribute__((always_inline)) {
        v += __uint_as_float(lane_xor<decltype(d)::value>(__float_as_uint(v)));
    });
    return v;
}

// LANES lanes a row, PER consecutive values each (E_n <= LANES PER), as keys in
// registers.  A round finds the largest key of a lane and of the lanes, and the
// first lane and place that hold it; a taken key becomes 0.  Lane j keeps the j-th
// choice (k <= LANES).  Few lanes a row cost few exchange steps.
template <typename E, int LANES, int PER>
__global__ __launch_bounds__(256) void route_kernel(const E *__restrict__ logits, int64_t ld, int64_t T, int En, int k,
                                                    bool sigmoid, bool renormalise, float scale,
                                                    int32_t *__restrict__ ids, float *__restrict__ w) {
    const int lane = threadIdx.x % LANES, group = threadIdx.x & 63 & ~(LANES - 1);
    const int64_t row = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    const int64_t t = row < T ? row : T - 1;  // whole wavefronts run; only rows of T are stored
    const E *p = logits + t * ld + lane * PER;
    const int have = En - lane * PER;
    float v[PER];
    if constexpr (PER * sizeof(E) % 16 == 0) {
        load_row(p, v, have);
    } else {
#pragma unroll
        for (int q = 0; q < PER; ++q) v[q] = q < have ? to_f32(p[q]) : 0.f;
    }
    uint32_t key[PER], top = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        key[q] = q < have && v[q] > -INFINITY ? order_key(v[q]) : 0;  // 0 for NaN too
        top = max(top, key[q]);
    }
    butterfly<LANES>([&](auto d) __attribute__((always_inline)) { top = max(top, lane_xor<decltype(d)::value>(top)); });
    const float largest = key_value(top);
    float sum = 0.f;
    if (!sigmoid) {  // exp(l - largest), 1 where l is the largest (also at +inf)
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (key[q] != 0) sum += key[q] == top ? 1.f : expf(v[q] - largest);
        sum = lane_sum<LANES>(sum);
    }
    uint32_t chosen = 0;
    int at = -1;
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int q = 1; q < PER; ++q) best = max(best, key[q]);
        uint32_t all = best;
        butterfly<LANES>([&](auto d) __attribute__((always_inline)) { all = max(all, lane_xor<decltype(d)::value>(all)); });
        // the first lane that holds it (lanes hold rising indices), and its first place
        const uint64_t holders = __ballot(best == all) >> group;
        const int first = __ffsll((unsigned long long)holders) - 1;
        int place = 0;
#pragma unroll
        for (int q = PER - 1; q >= 0; --q) place = key[q] == all ? q : place;
#pragma unroll
        for (int q = 0; q < PER; ++q) key[q] = lane == first && q == place ? 0 : key[q];
        const int index = __shfl(lane * PER + place, group + first);
        if (lane == j) {
            chosen = all;
            at = all != 0 ? index : -1;
        }
    }
    float weight = 0.f;
    if (at >= 0) {
        const float l = key_value(chosen);
        // The score.  To be renormalised a sigmoid of rows below 0 is taken relative to
        // the row's largest, s(l) / s(m) = exp(l - m) (1 + exp(m)) / (1 + exp(l)): below
        // -88 the scores themselves are 0 in float32, their ratios are not.
        if (!sigmoid) weight = (chosen == top ? 1.f : expf(l - largest)) / sum;
        else if (renormalise && largest < 0.f) weight = (chosen == top ? 1.f : expf(l - largest)) * (1.f + expf(largest)) / (1.f + expf(l));
        else weight = 1.f / (1.f + expf(-l));
    }
    if (renormalise) {
        const float total = lane_sum<LANES>(weight);
        if (total > 0.f) weight /= total;
    }
    if (row < T && lane < k) {
        ids[t * k + lane] = at;
        w[t * k + lane] = weight * scale;
    }
}

template <typename E, int LANES, int PER>
hipError_t launch_route_lanes(const E *logits, int64_t ld, int64_t T, int En, int k, bool sigmoid, bool renormalise,
                              float scale, int32_t *ids, float *w, hipStream_t st) {
    const int64_t grid = (T + 256 / LANES - 1) / (256 / LANES);
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((route_kernel<E, LANES, PER>), dim3((unsigned)grid), dim3(256), 0, st, logits, ld, T, En, k,
                       sigmoid, renormalise, scale, ids, w);
    return hipGetLastError();
}

// ------------------------------------------------------------------ expert layer

// The places of ids grouped by expert, in order, and cut into slots of at most
// SLOT pairs of one expert: slot s holds pairs list[first[s] .. + count[s]) of
// expert[s].  Every workgroup builds the same ones.
template <int MAXP, int SLOT> struct Slots {
    uint16_t list[MAXP], expert[MAXP], first[MAXP], count[MAXP];
    int n;

    // All kThreads threads; `scratch`: kMoeMaxExperts + MAXP ints of LDS; ends with
    // a barrier, or, up to 64 places, with every wavefront having written it all.
    // Places whose id is no expert are left out.
    __device__ __forceinline__ void build(const int32_t *ids, int places, int experts, int *scratch) {
        if (places <= 64) build_small(ids, places, experts);
        else build_any(ids, places, experts, scratch);
    }
    // The lanes whose id is this one's.
    static __device__ __forceinline__ uint64_t equals(int e, int bits) {
        uint64_t same = __ballot(e >= 0);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot(e >> b & 1);
            same &= e >> b & 1 ? set : ~set;
        }
        return same;
    }
    static __device__ __forceinline__ int id_bits(int experts) { return 32 - __clz((experts - 1) | 1); }
    // A place a lane, in registers, experts in the order of their first places: each
    // wavefront by itself, all write the same and none waits for another (1 token,
    // 128 experts, 8 places, 2048 x 768: the two kernels 15.4 + 10.2 us with the
    // other build alone).
    __device__ __forceinline__ void build_small(const int32_t *ids, int places, int experts) {
        const int lane = threadIdx.x & 63;
        const uint64_t below = (uint64_t{1} << lane) - 1;
        int e = lane < places ? ids[lane] : -1;
        e = e >= 0 && e < experts ? e : -1;
        const uint64_t same = equals(e, id_bits(experts));
        const int rank = __popcll(same & below);
        const bool leads = e >= 0 && rank == 0;
        const int c = leads ? __popcll(same) : 0, s = (c + SLOT - 1) / SLOT;
        // sums of pairs and slots over the leaders below, bit by bit
        int p0 = 0, s0 = 0, total = 0;
#pragma unroll
        for (int b = 0; b < 7; ++b) {
            p0 += __popcll(__ballot(c >> b & 1) & below) << b;
            if ((SLOT << b) <= 64 * 2) {
                const uint64_t m = __ballot(s >> b & 1);
                s0 += __popcll(m & below) << b;
                total += __popcll(m) << b;
            }
        }
        for (int q = 0; q < s; ++q) {
            expert[s0 + q] = (uint16_t)e;
            first[s0 + q] = (uint16_t)(p0 + SLOT * q);
            count[s0 + q] = (uint16_t)min(SLOT, c - SLOT * q);
        }
        const int from = __shfl(p0, e >= 0 ? __ffsll((unsigned long long)same) - 1 : 0);
        if (e >= 0) list[from + rank] = (uint16_t)lane;
        n = total;
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
        asm volatile("" ::: "memory");
    }
    __device__ __forceinline__ void build_any(const int32_t *ids, int places, int experts, int *scratch) {
        int *const cursor = scratch, *const id = scratch + kMoeMaxExperts;
        const int tid = threadIdx.x, lane = tid & 63;
        for (int e = tid; e < experts; e += kThreads) cursor[e] = 0;
        __syncthreads();
        for (int p = tid; p < places; p += kThreads) {
            const int e = ids[p];
            id[p] = e >= 0 && e < experts ? e : -1;
            if (id[p] >= 0) atomicAdd(&cursor[e], 1);
        }
        __syncthreads();
        if (tid < 64) {
            int pairs = 0, slots = 0;
            for (int e0 = 0; e0 < experts; e0 += 64) {
                const int e = e0 + lane;
                const int c = e < experts ? cursor[e] : 0, s = (c + SLOT - 1) / SLOT;
                int both = c | s << 16;  // prefix sums of pairs and slots (both below 2^15)
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    const int v = __shfl_up(both, d);
                    if (lane >= d) both += v;
                }
                const int p0 = pairs + (both & 0xffff) - c, s0 = slots + (both >> 16) - s;
                for (int q = 0; q < s; ++q) {
                    expert[s0 + q] = (uint16_t)e;
                    first[s0 + q] = (uint16_t)(p0 + SLOT * q);
                    count[s0 + q] = (uint16_t)min(SLOT, c - SLOT * q);
                }
                if (e < experts) cursor[e] = p0;
                const int last = __shfl(both, 63);
                pairs += last & 0xffff;
                slots += last >> 16;
            }
            if (lane == 0) n = slots;
            // 64 places at a time: a place's rank among those of its expert is the
            // number of equal ids in the lanes below, found by one ballot per bit
            const int bits = id_bits(experts);
            for (int p0 = 0; p0 < places; p0 += 64) {
                const int e = p0 + lane < places ? id[p0 + lane] : -1;
                const uint64_t same = equals(e, bits);
                if (e >= 0) {
                    const int rank = __popcll(same & ((uint64_t{1} << lane) - 1)), at = cursor[e];
                    list[at + rank] = (uint16_t)(p0 + lane);
                    if (rank == 0) cursor[e] = at + __popcll(same);
                }
            }
        }
        __syncthreads();
    }
};

// H = act(X Wg_e^T) * (X Wu_e^T) of every pair.  A unit is 8 gate and the same 8
// up rows of one slot's expert; a workgroup takes a contiguous run of units, slot
// by slot, so that a slot's tokens stay in registers over its units.
constexpr int kUpSlot = 32;
struct UpLds {
    StreamLds<2> stream;
    Slots<kMoeMaxPairs, kUpSlot> slots;
};
template <typename E> struct UpPosition {
    static constexpr int kFinishers = 8 * kUpSlot;
    const MoeArgs<E> *a;
    const Slots<kMoeMaxPairs, kUpSlot> *L;
    int tiles, left, slot, tile, pairs;
    int64_t row;  // of this tile in the stacked [experts * f] rows
    __device__ UpPosition(const MoeArgs<E> &args, const Slots<kMoeMaxPairs, kUpSlot> &slots) : a(&args), L(&slots) {
        tiles = (int)((a->f + 7) / 8);
        const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(L->n) * tiles;
        const int u0 = (int)(total * blockIdx.x / gridDim.x);
        left = (int)(total * (blockIdx.x + 1) / gridDim.x) - u0;
        slot = u0 / tiles;
        tile = u0 % tiles;
        enter();
        row += 8 * (int64_t)tile;
    }
    __device__ __forceinline__ void enter() {
        pairs = __builtin_amdgcn_readfirstlane(L->count[slot]);
        row = (int64_t)__builtin_amdgcn_readfirstlane(L->expert[slot]) * a->f;
    }
    __device__ __forceinline__ void advance() {
        row += 8;
        if (++tile == tiles) {
            tile = 0;
            ++slot;
            enter();
        }
    }
    __device__ __forceinline__ void weights(SlabRows &w, bool fresh) const {
        // rows past f are the next expert's or lie past the end of the buffer:
        // their products are not stored
        const int64_t bytes = ((int64_t)a->experts * a->f - row) * a->c * (int64_t)sizeof(E);
        w.buf[0] = panel(a->Wg + row * a->c, bytes);
        w.buf[1] = panel(a->Wu + row * a->c, bytes);
        if (!fresh) return;
#pragma unroll
        for (int q = 0; q < 2; ++q)
            w.off[q] = (uint32_t)(slab_row(q) & 7) * (uint32_t)(a->c * sizeof(E)) + slab_chunk();
    }
    __device__ __forceinline__ bool new_tokens() const { return tile == 0; }
    __device__ __forceinline__ int blocks() const { return pairs > 16 ? 2 : 1; }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t tokens() const { return panel(a->X); }
    __device__ __forceinline__ uint32_t token_row(int t) const {
        const int at = 16 * t + (threadIdx.x & 15);
        if (at >= pairs) return kOutside;
        return (uint32_t)(L->list[L->first[slot] + at] / a->k) * (uint32_t)(a->ldx * sizeof(E));
    }
    __device__ __forceinline__ void finish(const float *sums, int thread) const {
        const int q = thread & 7, at = thread >> 3;
        const int64_t c = 8 * (int64_t)tile + q;
        if (at >= pairs || c >= a->f) return;
        const float *block = sums + (at >> 4) * kWaves * kBlockSums;
        float y[1] = {joined(block, at & 15, q)};
        activate<sizeof(E) == 4>(y, a->act);
        const float h = y[0] * joined(block, at & 15, 8 + q);
        const int64_t pair = L->list[L->first[slot] + at];
        if constexpr (sizeof(E) == 2) {
            if (a->rest) {
                // the eight lanes of a pair hold its eight features: each stores one word of
                // the 32 bytes (two stores of half words: 8 us more at 48 tokens over 64
                // experts, as the ring waits for stores too).  Of an infinity nothing is left.
                const E high = to_elem<E>(h);
                const E low = to_elem<E>(fabsf(to_f32(high)) < INFINITY ? h - to_f32(high) : 0.f);
                const uint32_t both = __builtin_bit_cast(uint16_t, high) | (uint32_t)__builtin_bit_cast(uint16_t, low) << 16;
                const int from = (threadIdx.x & 56) + 2 * (q & 3);
                const uint32_t even = __shfl(both, from), odd = __shfl(both, from + 1);
                reinterpret_cast<uint32_t *>(a->H)[pair * a->f + c] =
                    q < 4 ? (even & 0xffff) | odd << 16 : even >> 16 | (odd & 0xffff0000);
                return;
            }
        }
        a->H[pair * a->f + c] = to_elem<E>(h);
    }
};

template <typename E, int SLABS> __global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs<E> a) {
    __shared__ __align__(16) UpLds lds;
    lds.slots.build(a.ids, a.T * a.k, a.experts, reinterpret_cast<int *>(lds.stream.ring));
    if (lds.slots.n == 0) return;
    const UpPosition<E> start(a, lds.slots);
    stream_products<E, SLABS, 2>(start, (int)(a.c * (int)sizeof(E)), lds.stream);
}

// Y = R + sum_j w_j H_j Wd_e^T.  A workgroup owns ROWS output features of a chunk
// of tokens.  The slabs of f of all its slots, one slot after the other, are
// dealt to its wavefronts in eight equal runs; a wavefront streams the weights'
// and the pairs' slabs of its run through its ring and keeps one slot's sums at a
// time.  A run's sums of a slot go to the pairs' own places in LDS, except
// those of a first slot that the run before began: these go to the wavefront's
// own place and are added afterwards in the order of the wavefronts.  At the end
// each token's places are added in order.
template <int ROWS, int SLOT> struct DownLds {
    char ring[kWaves * kRingBytes];
    float sums[down_pairs(ROWS) * ROWS];  // of every pair
    float head[kWaves][16 * ROWS];        // of a run's first slot, begun by the run before
    float weight[down_pairs(ROWS)];
    Slots<down_pairs(ROWS), SLOT> slots;
};
// Slots hold SLOT pairs: of 8, the ring holds more weights; of 16, an expert of
// more than 8 pairs is read once.  REST: H has two parts, which are rows 2 i and
// 2 i + 1 of the pairs' slabs, so that a copy reads whole lines; a pair's sum is
// that of two neighbouring lanes (16 tokens over 8 experts of 4096 x 14336, both
// kernels: 479 us; as rows i and 8 + i of separate buffers 486).
//
// Where c gives fewer workgroups than CUs, gridDim.z of them share the slabs of
// the same features, each dealing its part to its wavefronts as above, and leave
// the tokens' sums in `parts` for moe_join_kernel.
template <typename E, int ROWS, int SLOT, bool REST>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs<E> a, int chunk, float *parts) {
    __shared__ __align__(16) DownLds<ROWS, SLOT> lds;
    float *const P = lds.sums, *const weight = lds.weight;
    auto &L = lds.slots;
    auto &head = lds.head;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int t0 = (int)blockIdx.y * chunk, tn = min(chunk, a.T - t0), places = tn * a.k;
    const int64_t c0 = (int64_t)blockIdx.x * ROWS;
    const int32_t *ids = a.ids + (int64_t)t0 * a.k;
    for (int p = tid; p < places; p += kThreads) {
        const int e = ids[p];
        const bool chosen = e >= 0 && e < a.experts;
        weight[p] = chosen ? a.w[(int64_t)t0 * a.k + p] : 0.f;
        if (!chosen || parts) {  // adds 0, or what this workgroup has of it
#pragma unroll
            for (int q = 0; q < ROWS; ++q) P[p * ROWS + q] = 0.f;
        }
    }
    // the residual of this thread's first result, ahead of the stream
    float residual = 0.f;
    if (a.R && !parts && tid < tn * ROWS && c0 + tid % ROWS < a.c)
        residual = to_f32(a.R[(int64_t)(t0 + tid / ROWS) * a.ldr + c0 + tid % ROWS]);
    L.build(ids, places, a.experts, reinterpret_cast<int *>(lds.ring));
    const int row_bytes = (int)(a.f * (int)sizeof(E));
    const int slabs = (row_bytes + 127) / 128;
    const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(L.n) * slabs;
    const int runs = kWaves * (int)gridDim.z, run0 = kWaves * (int)blockIdx.z;
    auto run_start = [&](int v) { return total * (run0 + v) / runs; };
    if (parts) __syncthreads();  // the sums' zeros
    const int64_t r0 = run_start(wave), r1 = run_start(wave + 1);

    SlabRows w, x, x2;
    SlabRing<E, ROWS, REST ? 2 * SLOT : SLOT> ring{lds.ring + wave * kRingBytes};
    int64_t in_left = r1 - r0;
    int in_slot = (int)(r0 / slabs), in_slab = (int)(r0 % slabs);
    constexpr int WIDE = REST ? 2 : 1;  // H's row, in rows of Wd
    x.buf[0] = x.buf[1] = x2.buf[0] = x2.buf[1] = panel(a.H + (int64_t)t0 * a.k * a.f * WIDE);
    auto aim = [&]() __attribute__((always_inline)) {
        const int e = __builtin_amdgcn_readfirstlane(L.expert[in_slot]);
        w.buf[0] = w.buf[1] = panel(a.Wd + ((int64_t)e * a.c + c0) * a.f);
        const int last = (int)min((int64_t)ROWS, a.c - c0) - 1, n = L.count[in_slot], f0 = L.first[in_slot];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            w.off[q] = (uint32_t)min(slab_row(q), last) * (uint32_t)row_bytes + slab_chunk();
            // rows past the slot's pairs read nothing
            // REST: pairs 8 .. 15 in x2
            const int i = slab_row(q) / WIDE;
            const uint32_t in_row = WIDE * slab_chunk() + (REST ? 16 * (slab_row(q) & 1) : 0);
            x.off[q] = i < n ? (uint32_t)L.list[f0 + i] * (uint32_t)(WIDE * row_bytes) + in_row : kOutside;
            x2.off[q] = i + 8 < n ? (uint32_t)L.list[f0 + i + 8] * (uint32_t)(WIDE * row_bytes) + in_row : kOutside;
        }
    };
    auto ahead = [&]() __attribute__((always_inline)) {
        ring.issue(w, x, x2, 128u * (uint32_t)in_slab, 128u * WIDE * (uint32_t)in_slab, in_left > 0 ? row_bytes - 128 * in_slab : 0);
        --in_left;
        if (++in_slab == slabs) {
            in_slab = 0;
            ++in_slot;
            if (in_left > 0) aim();
        }
    };
    if (in_left > 0) aim();
    else w.buf[0] = w.buf[1] = x.buf[0];  // a run of nothing
#pragma unroll 1
    for (int p = 0; p < ring.DEPTH; ++p) ahead();

    int slot = (int)(r0 / slabs), slab = (int)(r0 % slabs);
    bool begun = slab != 0 && wave != 0;  // by the run before, of this workgroup
    f32x4 acc = {}, acc2 = {};
    // the pair of the slot whose sums this lane holds in the end
    const int mine = REST ? (i16 >> 1) + (SLOT == 16 ? 8 * (i16 & 1) : 0) : i16;
    const bool keeps = 4 * g < ROWS && (!REST || SLOT == 16 || i16 % 2 == 0);
#pragma unroll 1
    for (int64_t r = r0; r < r1; ++r) {
        SlabFrag<E> fw, fx, fx2;
        ring.take(fw, fx, fx2);
        ahead();
        acc = slab_product(acc, fw, fx);
        if constexpr (REST && SLOT == 16) acc2 = slab_product(acc2, fw, fx2);
        if (++slab == slabs || r + 1 == r1) {
            if constexpr (REST) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    acc[t] += __uint_as_float(lane_xor<1>(__float_as_uint(acc[t])));
                    if constexpr (SLOT == 16) {
                        acc2[t] += __uint_as_float(lane_xor<1>(__float_as_uint(acc2[t])));
                        acc[t] = i16 % 2 == 0 ? acc[t] : acc2[t];
                    }
                }
            }
            if (keeps) {
                if (begun) *reinterpret_cast<f32x4 *>(&head[wave][mine * ROWS + 4 * g]) = acc;
                else if (mine < L.count[slot])
                    *reinterpret_cast<f32x4 *>(&P[L.list[L.first[slot] + mine] * ROWS + 4 * g]) = acc;
            }
            acc = acc2 = f32x4{};
            begun = false;
            slab = 0;
            ++slot;
        }
    }
    wait_vmcnt<0>();
    __syncthreads();
    if (tid < 16 * ROWS) {  // this thread's column and row of every slot that a run continued
        const int i = tid / ROWS, q = tid % ROWS;
        for (int v = 1; v < kWaves; ++v) {
            const int64_t b = run_start(v);
            const int s = (int)(b / slabs);
            if (b < run_start(v + 1) && b % slabs != 0 && i < L.count[s])
                P[L.list[L.first[s] + i] * ROWS + q] += head[v][i * ROWS + q];
        }
    }
    __syncthreads();
    for (int u = tid; u < tn * ROWS; u += kThreads) {
        const int t = u / ROWS, q = u % ROWS;
        const int64_t tok = t0 + t;
        if (c0 + q >= a.c) continue;
        float sum = 0.f;
        for (int j = 0; j < a.k; ++j) sum += weight[t * a.k + j] * P[(t * a.k + j) * ROWS + q];
        if (parts) {
            parts[((int64_t)blockIdx.z * a.T + tok) * a.c + c0 + q] = sum;
            continue;
        }
        if (u < kThreads) sum += residual;
        else if (a.R) sum += to_f32(a.R[tok * a.ldr + c0 + q]);
        a.Y[tok * a.ldy + c0 + q] = to_elem<E>(sum);
    }
}

// Y = R + the parts of every token, in their order; four columns a thread.
template <typename E>
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs<E> a, const float *__restrict__ parts, int splits) {
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x, quads = a.c / 4;
    if (u >= a.T * quads) return;
    const int64_t t = u / quads, c = 4 * (u - t * quads);
    f32x4 sum = {};
#pragma unroll 4
    for (int z = 0; z < splits; ++z) sum += *reinterpret_cast<const f32x4 *>(parts + (z * (int64_t)a.T + t) * a.c + c);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        a.Y[t * a.ldy + c + q] = to_elem<E>(sum[q] + (a.R ? to_f32(a.R[t * a.ldr + c + q]) : 0.f));
}

template <typename E, int SLABS> hipError_t launch_up(const MoeArgs<E> &a, hipStream_t st) {
    const int64_t most = (int64_t)std::min(a.T * a.k, a.experts + a.T * a.k / 32) * ((a.f + 7) / 8);  // units
    hipLaunchKernelGGL((moe_up_kernel<E, SLABS>), dim3((unsigned)std::min<int64_t>(most, 256)), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}
template <typename E, int ROWS, int SLOT, bool REST> hipError_t launch_down(const MoeArgs<E> &a, hipStream_t st) {
    const int chunk = std::min(a.T, down_pairs(ROWS) / a.k);
    const int64_t rows = (a.c + ROWS - 1) / ROWS, chunks = (a.T + chunk - 1) / chunk;
    const int splits = down_splits({ROWS, SLOT}, sizeof(E), a.T, a.k, a.experts, a.c, a.f, a.parts != nullptr, REST);
    const bool split = splits > 1;
    hipLaunchKernelGGL((moe_down_kernel<E, ROWS, SLOT, REST>), dim3((unsigned)rows, (unsigned)chunks, (unsigned)splits),
                       dim3(kThreads), 0, st, a, chunk, split ? a.parts : nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !split) return e;
    hipLaunchKernelGGL((moe_join_kernel<E>), dim3((unsigned)((a.T * (a.c / 4) + 255) / 256)), dim3(256), 0, st, a, a.parts,
                       splits);
    return hipGetLastError();
}

}  // namespace

template <typename E>
hipError_t launch_route(const E *logits, int64_t ld, int64_t T, int En, int k, bool sigmoid, bool renormalise,
                        float scale, int32_t *ids, float *w, hipStream_t st) {
    if (T <= 0) return hipSuccess;
    // 16 lanes a row where they hold its values (up to 16 each) and its choices
#define DYRA_ROUTE(LANES, PER) \
    launch_route_lanes<E, LANES, PER>(logits, ld, T, En, k, sigmoid, renormalise, scale, ids, w, st)
    if (k <= 16 && En <= 256)
        return En <= 32 ? DYRA_ROUTE(16, 2) : En <= 64 ? DYRA_ROUTE(16, 4) : En <= 128 ? DYRA_ROUTE(16, 8) : DYRA_ROUTE(16, 16);
    return En <= 256 ? DYRA_ROUTE(64, 4) : En <= 512 ? DYRA_ROUTE(64, 8) : DYRA_ROUTE(64, 16);
#undef DYRA_ROUTE
}

template <typename E> hipError_t launch_moe(const MoeArgs<E> &a, hipStream_t st) {
    if (a.T <= 0) return hipSuccess;
    if (a.T * a.k > kMoeMaxPairs || a.experts > kMoeMaxExperts) return hipErrorInvalidValue;
    static_assert(kWaves == 8, "up_slabs divides c by it");
    const int slabs = up_slabs(a.c * (int64_t)sizeof(E));
    const hipError_t e = slabs == 2   ? launch_up<E, 2>(a, st)
                         : slabs == 4 ? launch_up<E, 4>(a, st)
                         : slabs == 8 ? launch_up<E, 8>(a, st)
                                      : launch_up<E, 12>(a, st);
    if (e != hipSuccess) return e;
    const Down d = down_kernel(a.T, a.k, a.experts, a.c);
    auto go = [&](auto rest) {
        constexpr bool REST = decltype(rest)::value;
        if (d.rows == 8) return d.slot == 8 ? launch_down<E, 8, 8, REST>(a, st) : launch_down<E, 8, 16, REST>(a, st);
        return d.slot == 8 ? launch_down<E, 16, 8, REST>(a, st) : launch_down<E, 16, 16, REST>(a, st);
    };
    if constexpr (sizeof(E) == 2) {
        if (a.rest) return go(std::true_type{});
    }
    return go(std::false_type{});
}

template hipError_t launch_route<float>(const float *, int64_t, int64_t, int, int, bool, bool, float, int32_t *, float *,
                                        hipStream_t);
template hipError_t launch_route<bf16>(const bf16 *, int64_t, int64_t, int, int, bool, bool, float, int32_t *, float *,
                                       hipStream_t);
template hipError_t launch_moe<float>(const MoeArgs<float> &, hipStream_t);
template hipError_t launch_moe<bf16>(const MoeArgs<bf16> &, hipStream_t);

}  // namespace dyra
