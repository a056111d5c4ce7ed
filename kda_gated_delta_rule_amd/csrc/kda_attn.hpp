// kda_attn.hpp -- tile primitives of the softmax-attention kernels (prompt forward and backward):
// 32x32 MFMA fragments, swizzled LDS tiles and the map from workgroups to packed sequences.
#pragma once

#include "kda_device.hpp"

namespace kda {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// 32x32 output tiles, 16 k elements per step.  Lane l (r = l % 32, h = l / 32) supplies eight
// elements of row r of each operand; which k they are does not matter as long as both operands
// agree.  Two orders are used:
//   row order   k = k0 + 8h + j                      (16 or 32 contiguous bytes of an LDS row)
//   acc order   k = k0 + 4h + j, j < 4; k0 + 8 + 4h + j - 4 above
// The accumulator holds C[8 (i / 4) + 4h + i % 4][r] in element i, so elements 8s .. 8s + 7 of one
// product are, in acc order, the k step s of the next product's B operand with no exchange of lanes.
//   bf16: one v_mfma_f32_32x32x16_bf16;  fp32: eight v_mfma_f32_32x32x2_f32, step j taking the
//   j-th element of both halves.
// ---------------------------------------------------------------------------
template <class T>
struct Frag;
template <>
struct Frag<BF16> {
    bf16x8 v;
};
template <>
struct Frag<F32> {
    float v[8];
};

__device__ __forceinline__ f32x16 mma32(const Frag<BF16>& a, const Frag<BF16>& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(const Frag<F32>& a, const Frag<F32>& b, f32x16 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b.v[j], c, 0, 0, 0);
    return c;
}

// Elements 8s .. 8s + 7 of an accumulator as a B operand (bf16: rounded to nearest even).
template <class T>
__device__ __forceinline__ Frag<T> frag_from_acc(const f32x16& c, int s);
template <>
__device__ __forceinline__ Frag<BF16> frag_from_acc<BF16>(const f32x16& c, int s) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(c[8 * s + 2 * j], c[8 * s + 2 * j + 1]);
    Frag<BF16> f;
    f.v = __builtin_bit_cast(bf16x8, w);
    return f;
}
template <>
__device__ __forceinline__ Frag<F32> frag_from_acc<F32>(const f32x16& c, int s) {
    Frag<F32> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = c[8 * s + j];
    return f;
}

// Eight contiguous elements in global memory (16-byte aligned), negated when neg.
__device__ __forceinline__ Frag<BF16> frag_load(const uint16_t* p, bool neg) {
    u32x4 w = *reinterpret_cast<const u32x4*>(p);
    w ^= neg ? 0x80008000u : 0u;
    Frag<BF16> f;
    f.v = __builtin_bit_cast(bf16x8, w);
    return f;
}
__device__ __forceinline__ Frag<F32> frag_load(const float* p, bool neg) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    Frag<F32> f = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    if (neg)
#pragma unroll
        for (int j = 0; j < 8; ++j) f.v[j] = -f.v[j];
    return f;
}

// ---------------------------------------------------------------------------
// LDS tile of ROWS rows of D elements.  The 16-byte chunk c of a row is kept at place c ^ swz(row).
// Rows at one chunk (row fragments, 16 lanes a pass) then spread over all 64 banks, and so do four
// rows of the 64 bytes that a transposed read takes.
// ---------------------------------------------------------------------------
template <class T, int D>
struct Tile {
    using elem = typename T::storage;
    static constexpr int kChunks = D * T::bytes / 16;  // per row
    static constexpr int kPer = 16 / T::bytes;         // elements of a chunk
    static constexpr int kRowBytes = D * T::bytes;

    __device__ static __forceinline__ int swz(int row) {
        if (kChunks >= 16) return ((row & 3) << 2) | ((row >> 2) & 3);
        // 128-byte rows: two rows share the 256 bytes of the banks
        return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
    }
    __device__ static __forceinline__ int at(int row, int chunk) {  // byte offset
        return row * kRowBytes + ((chunk ^ swz(row)) << 4);
    }

    // Row fragment (row order): elements k0 + 8h .. + 7 of row.
    __device__ static __forceinline__ Frag<T> row_frag(const char* tile, int row, int k0, int h) {
        Frag<T> f;
        if constexpr (T::bytes == 2) {
            f.v = *reinterpret_cast<const bf16x8*>(tile + at(row, k0 / 8 + h));
        } else {
            const float4 a = *reinterpret_cast<const float4*>(tile + at(row, k0 / 4 + 2 * h));
            const float4 b = *reinterpret_cast<const float4*>(tile + at(row, k0 / 4 + 2 * h + 1));
            f.v[0] = a.x, f.v[1] = a.y, f.v[2] = a.z, f.v[3] = a.w;
            f.v[4] = b.x, f.v[5] = b.y, f.v[6] = b.z, f.v[7] = b.w;
        }
        return f;
    }

    // Transposed fragment (acc order): column d0 + lane % 32 of rows k0 .. k0 + 15.  bf16: a
    // transposing LDS read gives lane i of each 16 lanes column i of the four rows that the 16
    // lanes point at, four lanes (8 bytes each) a row.
    __device__ static __forceinline__ Frag<T> col_frag(const char* tile, int k0, int d0, int lane) {
        const int h = lane >> 5;
        Frag<T> f;
        if constexpr (T::bytes == 2) {
            const int i = lane & 15, row = k0 + 4 * h + (i >> 2);
            const int col = d0 + 16 * ((lane >> 4) & 1) + 4 * (i & 3);
            using lds = __attribute__((address_space(3))) s16x4;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds*)(tile + at(row, col >> 3) + 2 * (col & 4)));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds*)(tile + at(row + 8, col >> 3) + 2 * (col & 4)));
            f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int col = d0 + (lane & 31);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int row = k0 + 4 * h + (j < 4 ? j : j + 4);
                f.v[j] = *reinterpret_cast<const float*>(tile + at(row, col >> 2) + 4 * (col & 3));
            }
        }
        return f;
    }
};

// Workgroup barrier behind which every wave's tile copies (counted as global loads) and LDS accesses
// are done.
__device__ __forceinline__ void tile_barrier() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Wave-wide copy of a tile from global memory into LDS, 16 bytes a lane, without registers: a load
// puts lane l's chunk at LDS address base + 16 l, so the swizzle is applied to the global side.
// The compiler does not wait for the copy at LDS reads through pointers that it knows to be others
// (restrict arguments of an inlined function), nor does __syncthreads(): tile_barrier() does.
template <class T, int D, int ROWS, int NT>
struct Copy {
    using TL = Tile<T, D>;
    static constexpr int kN = ROWS * TL::kChunks / NT;  // chunks of a thread
    static constexpr int kStep = NT / TL::kChunks;      // rows between them
    static constexpr int kP = kStep % 16 ? 16 / kStep : 1;  // after so many the swizzle is the first's again
    static_assert(ROWS * TL::kChunks % NT == 0 && NT % TL::kChunks == 0 && 16 % kP == 0, "whole chunks per thread");
    int off[kP];  // bytes from the tile's first row
    int ld;       // bytes of a row stride (host-checked: 2^24 at most)

    __device__ __forceinline__ int place(int i, int tid, int last) const {
        const int n = i * NT + tid, row = n / TL::kChunks;
        return min(row, last) * ld + ((n % TL::kChunks ^ TL::swz(row)) << 4);
    }
    __device__ __forceinline__ Copy(int64_t ld_elems, int tid)
        : ld(__builtin_amdgcn_readfirstlane(static_cast<int>(ld_elems * T::bytes))) {
#pragma unroll
        for (int i = 0; i < kP; ++i) off[i] = place(i, tid, ROWS);
    }
    // Rows row0 .. row0 + ROWS - 1 of base; those past row `last` repeat it, so that nothing outside
    // the sequence is read.
    __device__ __forceinline__ void start(const typename T::storage* base, int row0, int last, char* tile, int tid,
                                          int wave) const {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass has no type for a buffer resource
        const char* p = reinterpret_cast<const char*>(base) + static_cast<int64_t>(row0) * ld;
        const int left = min(last - row0, ROWS - 1);
        const auto rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, left * ld + TL::kRowBytes, 0x00020000);
        const auto copy = [&](int i, int from, int more) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void*)(tile + (i * NT + wave * kWave) * 16), 16, from, more,
                0, 0);
        };
        if (left == ROWS - 1) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                copy(i, off[i % kP], __builtin_amdgcn_readfirstlane(i / kP * kP * kStep * ld));
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) copy(i, place(i, tid, left), 0);
        }
#endif
    }
};

// Order of a block of LDS reads and the bf16 MFMAs that take them: READS reads for every MFMA, the
// first AHEAD MFMAs' (and MORE others) before them, so that a read's latency (about 130 cycles, four
// MFMAs) is behind it when its MFMA comes.  Left alone, the compiler puts a read right before its
// MFMA.
template <class T, int MFMAS, int READS, int AHEAD, int MORE = 0>
__device__ __forceinline__ void read_ahead() {
    if constexpr (T::bytes == 2) {
        __builtin_amdgcn_sched_group_barrier(0x100, READS * AHEAD + MORE, 0);
#pragma unroll
        for (int i = 0; i < MFMAS - AHEAD; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, AHEAD, 0);
    }
}

// Value of the other half-wave's lane with the same lane % 32.
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, kWave); }

// ---------------------------------------------------------------------------
// Packed sequences.  A sequence's tokens are cu[i] .. cu[i + 1] - 1, kept within 0 .. total so
// that a wrong cu_seqlens reads and writes nothing outside the arrays.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int seq_bound(const int32_t* cu, int i, int total) { return min(max(cu[i], 0), total); }

// Inclusive prefix sum over the wave's lanes (row shifts, then the rows' last lanes onward).
__device__ __forceinline__ int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
    return x;
}
__device__ __forceinline__ int wave_total(int x) { return __builtin_amdgcn_readlane(wave_scan(x), kWave - 1); }

// The same for a sum of floats, in one order for every wave, and for a maximum of ints above 0.
__device__ __forceinline__ float wave_total(float x) {
#define KDA_ROW_ADD(ctrl, rows) \
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), ctrl, rows, 0xf, false))
    KDA_ROW_ADD(0x111, 0xf);
    KDA_ROW_ADD(0x112, 0xf);
    KDA_ROW_ADD(0x114, 0xf);
    KDA_ROW_ADD(0x118, 0xf);
    KDA_ROW_ADD(0x142, 0xa);
    KDA_ROW_ADD(0x143, 0xc);
#undef KDA_ROW_ADD
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), kWave - 1));
}
__device__ __forceinline__ int wave_max(int x) {
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));
    return __builtin_amdgcn_readlane(x, kWave - 1);
}

// The lane and the rest of t in a row of counts n over the lanes: {lane, t - counts before it}, or
// {-1, t - all counts}.
__device__ __forceinline__ int2 find_in(int n, int t) {
    const int sum = wave_scan(n);
    const uint64_t past = __ballot(sum > t);
    if (!past) return make_int2(-1, t - __builtin_amdgcn_readlane(sum, kWave - 1));
    const int l = __ffsll(static_cast<unsigned long long>(past)) - 1;
    return make_int2(l, t - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(n, l)));
}

constexpr int kTileRows = 128;   // queries or keys of a workgroup
constexpr int kWorkUnit = 32;    // work of a tile is counted in this many of its counterparts
constexpr int kMaxParts = 1024;  // workgroups that share tiles, in all
constexpr int kMaxSplits = 16;   // workgroups that share one tile
constexpr float kLevel = 0.7f;   // most of a part, in even shares

// What a workgroup does: a tile of a sequence for one head, or one of `splits` equal parts of the
// counterparts that the tile goes through, whose sums go to place `part` of the workspace.
struct WorkItem {
    int seq;  // -1: nothing
    int tile;
    int head;  // its place in launch order
    int split, splits, part;
    int q0, Lq, k0, Lk;  // the sequence's queries and keys
};

// How the work is cut, the same in every workgroup of a launch.
//
// Causal tiles differ in work by the length of the sequence.  Up to 64 sequences (a lane each) are
// gone through by work, most first, so that a workgroup that starts late has little to do; tile j
// (of the queries: from the last, of the keys: from the first) has min(cap, max(A - 4 j, 0)) units,
// A from the keys, cap from the queries that there are to see them.  More than 64 sequences go in
// their order, unshared: of documents of 100 tokens and one of 8192 behind them, 8 heads on 1 of 128 in
// bf16, gradients take 585 us with 64 sequences and 1770 with 65 (32 heads on 8: 1925 and 1900, which
// fill the card by themselves; the forward 191 and 191, 597 and 583).
//
// With SPLIT, where a tile has more than an even share of the whole among `slots` workgroups (and more
// than `least` units, below which a part is not worth its sum), every tile of more than `level`
// units, 0.7 of an even share, is cut into ceil(units / level) equal parts: `heavy` tiles and `parts`
// parts for each head, max_parts in all at most, which the workspace has room for (else, seldom, with
// a whole share as the level).  Parts by a tile's own work, not as many for each: their sums are
// memory traffic (16 heads on 4 of 128, 700 to 2000 tokens, bf16: gradients 192 -> 181 us; one head
// of 8192: 155 -> 138, four on one 382 -> 328).  The level, in even shares: those gradients take 183 us
// with 0.6, 0.7 and 0.85, 187 with 1 and 198 with 0.5; fp32 prompts of 1501 and 700 with 16 heads of
// 64 take 90 us with 0.7, 95 with 1 and 98 with the others, where a last few parts start late.
template <bool KEYS, bool SPLIT>
struct WorkPlan {
    int q0 = 0, lq = 0, k0 = 0, lk = 0;  // the lane's sequence
    int n = 0, A = 0, cap = 0, top = 0;
    int lane, level = 0, heavy = 0, parts = 0;
    // lane j: shared tiles in exactly, and in more than, most - j parts
    int most = 1, exact = 0, beyond = 0;

    // Tiles of c units or more, of one sequence.
    __device__ static __forceinline__ int above(int c, int n, int A, int cap) {
        return c <= 0 ? n : c > cap || c > A ? 0 : min((A - c) / 4 + 1, n);
    }
    __device__ __forceinline__ int above(int c) const { return above(c, n, A, cap); }
    __device__ __forceinline__ WorkPlan(const int32_t* cu_q, const int32_t* cu_k, int num_seqs, int total_q,
                                        int total_k, int heads, int slots, int least, int max_parts, int l)
        : lane(l) {
        if (num_seqs > kWave) return;
        if (lane < num_seqs) {
            q0 = seq_bound(cu_q, lane, total_q), k0 = seq_bound(cu_k, lane, total_k);
            lq = max(seq_bound(cu_q, lane + 1, total_q) - q0, 0);
            lk = max(seq_bound(cu_k, lane + 1, total_k) - k0, 0);
            n = ((KEYS ? lk : lq) + kTileRows - 1) / kTileRows;
            A = (lk + kWorkUnit - 1) / kWorkUnit;
            cap = KEYS ? (lq + kWorkUnit - 1) / kWorkUnit : A;
        }
        top = wave_max(min(A, cap));
        if constexpr (SPLIT) {
            // sum over j < n of min(cap, max(A - 4 j, 0)): m tiles with work, c1 of them capped
            const int m = min(n, (A + 3) / 4), c1 = min(max((A - cap + 3) / 4, 0), m);
            const float fm = static_cast<float>(m), f1 = static_cast<float>(c1);
            const float sum = f1 * static_cast<float>(cap) +
                              (fm - f1) * (static_cast<float>(A) - 2.f * (fm + f1 - 1.f));
            const float even = fminf(wave_total(sum) * static_cast<float>(heads) / static_cast<float>(slots), 1e9f);
            const int share = max(__builtin_amdgcn_readfirstlane(static_cast<int>(even)) + 1, least);
            if (top > share) {
                level = max(__builtin_amdgcn_readfirstlane(static_cast<int>(kLevel * even)) + 1, least);
                count(heads, max_parts);
                if (heavy == 0 && level < share) level = share, count(heads, max_parts);
            }
        }
    }
    // The tiles shared at this level, none if their parts are too many: lane j counts those in most - j
    // parts or more over the sequences that have any.
    __device__ __forceinline__ void count(int heads, int max_parts) {
        most = min((top + level - 1) / level, kMaxSplits);
        const int s = most - lane;
        const int least = s >= 2 ? (s - 1) * level + 1 : INT32_MAX;
        const int more = s >= 2 && lane > 0 ? least + level : INT32_MAX;
        int reach = 0;
        beyond = 0;
        for (uint64_t big = __ballot(min(A, cap) > level); big; big &= big - 1) {
            const int i = __ffsll(static_cast<unsigned long long>(big)) - 1;
            const int tn = __builtin_amdgcn_readlane(n, i), tA = __builtin_amdgcn_readlane(A, i);
            const int tc = __builtin_amdgcn_readlane(cap, i);
            reach += above(least, tn, tA, tc), beyond += above(more, tn, tA, tc);
        }
        heavy = __builtin_amdgcn_readlane(reach, most - 2);
        exact = reach - beyond;
        parts = wave_total(exact * (most - lane));
        if (static_cast<int64_t>(parts) * heads > max_parts) heavy = parts = exact = 0;
    }

    // Parts of the shared tile of rank t: their number, and the place of the first among one head's.
    __device__ __forceinline__ int2 parts_of(int t) const {
        const int n = exact * (most - lane);
        const int2 at = find_in(exact, t);
        const int s = most - at.x;
        return make_int2(__builtin_amdgcn_readfirstlane(s),
                         __builtin_amdgcn_readlane(wave_scan(n) - n, at.x) + at.y * s);
    }

    // Tile of rank t by work.
    __device__ __forceinline__ void tile_of(int t, const int32_t* cu_q, const int32_t* cu_k, int num_seqs,
                                            int total_q, int total_k, WorkItem& w) const {
        const int32_t* cu = KEYS ? cu_k : cu_q;
        const int total = KEYS ? total_k : total_q;
        int seq = -1, tile = 0, tiles = 0;
        if (num_seqs <= kWave) {
            int lo = 0, hi = top + 1;  // tiles of lo units or more reach past t, of hi or more do not
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (wave_total(above(mid)) > t)
                    lo = mid;
                else
                    hi = mid;
            }
            const int more = above(lo + 1);
            const int2 at = find_in(above(lo) - more, t - wave_total(more));
            if (at.x >= 0) {
                seq = at.x;
                tile = __builtin_amdgcn_readlane(more, at.x) + at.y;
                tiles = __builtin_amdgcn_readlane(n, at.x);
                w.q0 = __builtin_amdgcn_readlane(q0, at.x), w.Lq = __builtin_amdgcn_readlane(lq, at.x);
                w.k0 = __builtin_amdgcn_readlane(k0, at.x), w.Lk = __builtin_amdgcn_readlane(lk, at.x);
            }
        } else {
            for (int base = 0; base < num_seqs && seq < 0; base += kWave) {
                const int i = base + lane;
                int c = 0;
                if (i < num_seqs)
                    c = (max(seq_bound(cu, i + 1, total) - seq_bound(cu, i, total), 0) + kTileRows - 1) / kTileRows;
                const int2 at = find_in(c, t);
                t = at.y;
                if (at.x >= 0) seq = base + at.x, tile = at.y, tiles = __builtin_amdgcn_readlane(c, at.x);
            }
            if (seq >= 0) {
                w.q0 = seq_bound(cu_q, seq, total_q), w.k0 = seq_bound(cu_k, seq, total_k);
                w.Lq = max(seq_bound(cu_q, seq + 1, total_q) - w.q0, 0);
                w.Lk = max(seq_bound(cu_k, seq + 1, total_k) - w.k0, 0);
            }
        }
        // the same in every lane, which addresses of scalar operands need to be known for
        const auto same = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
        w.seq = same(seq);
        w.tile = same(KEYS ? tile : tiles - 1 - tile);
        w.q0 = same(w.q0), w.Lq = same(w.Lq), w.k0 = same(w.k0), w.Lk = same(w.Lk);
    }

    // Workgroup `block` of a launch: the parts of the heavy tiles first, the heads of a tile together.
    __device__ __forceinline__ WorkItem item(int block, int heads, const int32_t* cu_q, const int32_t* cu_k,
                                             int num_seqs, int total_q, int total_k) const {
        WorkItem w{-1, 0, block % heads, 0, 1, block, 0, 0, 0, 0};
        int t = block / heads;
        if (SPLIT && t < parts) {
            const int2 at = find_in(exact * (most - lane), t);
            const int splits = __builtin_amdgcn_readfirstlane(most - at.x);
            const int place = __builtin_amdgcn_readfirstlane(at.y), tile = place / splits;
            w.splits = splits, w.split = place - tile * splits;
            t = __builtin_amdgcn_readlane(beyond, at.x) + tile;
        } else {
            t -= parts - heavy;
        }
        tile_of(t, cu_q, cu_k, num_seqs, total_q, total_k, w);
        return w;
    }
};

// The same from the host's side, which knows no lengths: whether a launch can have tiles to share,
// and the most parts that it can make.
inline bool work_may_split(int num_seqs, int64_t counterparts, int least) {
    return num_seqs <= kWave && counterparts > static_cast<int64_t>(kWorkUnit) * least;
}
inline int64_t work_tiles(int64_t total, int num_seqs, int heads) { return (total / kTileRows + num_seqs) * heads; }
inline int64_t work_parts(int64_t tiles) {
    return tiles * kMaxSplits < kMaxParts ? tiles * kMaxSplits : kMaxParts;
}

// Head of place p of H in a launch order: workgroups go to the eight XCDs in turn, so with H a
// multiple of 8 neighbouring heads (which share a kv head) meet in one XCD's L2.
__device__ __forceinline__ int head_of(int p, int H) { return (H & 7) ? p : (p & 7) * (H >> 3) + (p >> 3); }

}  // namespace kda
