// kda_attn_cache.hip -- the paged cache held in 8 bits, and the attention that decodes over it.
//
// A page holds block_tokens tokens of one sequence for every kv head, as e4m3 numbers times one
// power of two per (page, head): k_cache [page][Hk][token][dk], v_cache [page][Hk][dv][token]
// (turned, so that the product with the weights reads its k axis, the tokens, contiguously).
// Powers of two make every product with a scale exact, and moving a page to a larger scale loses
// nothing but bits below the smallest normal e4m3 number.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "kda_attn.hpp"
#include "kda_attn_plan.hpp"
#include "kda_internal.hpp"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kExpMin = -100, kExpMax = 120;  // of a page's scale

__device__ __forceinline__ float pow2(int e) {
    return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}
__device__ __forceinline__ int exp_of(float scale) {
    return min(max(static_cast<int>(__float_as_uint(scale) >> 23 & 255) - 127, kExpMin), kExpMax);
}

// The least e with amax <= 448 2^e (448 = 1.75 2^8), within kExpMin .. kExpMax.
__device__ __forceinline__ int cache_exp(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);
    return min(max(e, kExpMin), kExpMax);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}
// Four e4m3 numbers times f, rounded to e4m3 again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float f) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    return to_e4m3x4(lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f);
}

struct AppendBlock {
    int seq;     // -1: none
    int block;   // of the sequence
    int start;   // tokens the sequence held
    int len;     // tokens that join
    int tok0;    // the first of them in k and v
};

// Block t of those that the call writes into: every sequence with new tokens has
// ceil((start % bt + len) / bt) of them.
__device__ __forceinline__ AppendBlock find_block(const AttnAppendArgs& a, int t, int lane) {
    for (int base = 0; base < a.N; base += kWave) {
        const int i = base + lane;
        int n = 0;
        if (i < a.N) {
            const int len = seq_bound(a.cu, i + 1, a.total) - seq_bound(a.cu, i, a.total);
            const int in = max(a.start_len[i], 0) & (a.bt - 1);
            if (len > 0) n = (in + len + a.bt - 1) / a.bt;
        }
        const int2 at = find_in(n, t);
        t = at.y;
        if (at.x >= 0) {
            const int seq = base + at.x, tok0 = seq_bound(a.cu, seq, a.total), start = max(a.start_len[seq], 0);
            return {seq, start / a.bt + at.y, start, seq_bound(a.cu, seq + 1, a.total) - tok0, tok0};
        }
    }
    return {-1, 0, 0, 0, 0};
}

// A workgroup for each page that the call writes into, kv head, and k or v: it alone knows the page's
// largest value, and a page's scale and bytes have one writer.  128,076 tokens of 8 heads, 128 + 128,
// from bf16: 154-170 us, 4.6-5.1 TB/s of the bytes read and written, a large copy's rate (4.9).
// 64 sequences of one token: 8 us, the chain from the lengths over the table to the page; 12 us where half
// of the pages raise their scale, whose older numbers go through the registers again.
//
// One page and kv head of k (TURNED false) or v (true).  The new rows stay in registers between
// the search for their largest value and their conversion.
template <class T, int D, int BT, bool TURNED>
__device__ __forceinline__ void append_page(const AttnAppendArgs& a, const AppendBlock& b, int page, int head,
                                            char* lds, float* wave_max) {
    using E = typename T::storage;
    constexpr int kUnits = BT * D / 8, kPer = (kUnits + kThreads - 1) / kThreads;  // of eight values
    const int tid = threadIdx.x, pos0 = b.block * BT;
    const int64_t past = static_cast<int64_t>(b.start) + b.len - pos0;
    const int t0 = max(b.start - pos0, 0), t1 = static_cast<int>(min(static_cast<int64_t>(BT), past));
    const int64_t ld = TURNED ? a.ldv : a.ldk;
    const E* rows = static_cast<const E*>(TURNED ? a.v : a.k) + head * D;
    const int64_t at = static_cast<int64_t>(page) * a.Hk + head;
    uint8_t* cache = (TURNED ? a.v_cache : a.k_cache) + at * BT * D;
    float* scale = (TURNED ? a.v_scale : a.k_scale) + at;

    float x[kPer][8];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int u = i * kThreads + tid, pos = u / (D / 8), c = u % (D / 8);
        if (u < kUnits && pos >= t0 && pos < t1) {
            const int64_t tok = b.tok0 + (pos0 + pos - b.start);
            const float4 lo = load4<T>(rows, tok * ld + 8 * c), hi = load4<T>(rows, tok * ld + 8 * c + 4);
            x[i][0] = lo.x, x[i][1] = lo.y, x[i][2] = lo.z, x[i][3] = lo.w;
            x[i][4] = hi.x, x[i][5] = hi.y, x[i][6] = hi.z, x[i][7] = hi.w;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = fabsf(x[i][j]);
                if (m < INFINITY) amax = fmaxf(amax, m);
                else x[i][j] = NAN;  // e4m3 has no infinity
            }
        }
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m, kWave));
    if ((tid & 63) == 0) wave_max[tid >> 6] = amax;
    const int e_old = t0 > 0 ? exp_of(*scale) : kExpMin;
    __syncthreads();
    amax = fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
    const int e = max(cache_exp(amax), e_old);
    const float f = pow2(-e), f_old = pow2(e_old - e);
    const bool grown = t0 > 0 && e > e_old;
    if (tid == 0 && (t0 == 0 || grown)) *scale = pow2(e);

#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int u = i * kThreads + tid, pos = u / (D / 8), c = u % (D / 8);
        if (u >= kUnits) continue;
        if (pos >= t0 && pos < t1) {
            const uint32_t lo = to_e4m3x4(x[i][0] * f, x[i][1] * f, x[i][2] * f, x[i][3] * f);
            const uint32_t hi = to_e4m3x4(x[i][4] * f, x[i][5] * f, x[i][6] * f, x[i][7] * f);
            if constexpr (TURNED) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    lds[(8 * c + j) * (BT + 4) + pos] = static_cast<char>((j < 4 ? lo : hi) >> 8 * (j & 3));
            } else {
                *reinterpret_cast<uint2*>(cache + pos * D + 8 * c) = make_uint2(lo, hi);
            }
        } else if (!TURNED && pos < t0) {
            if (!grown) continue;
            uint2* p = reinterpret_cast<uint2*>(cache + pos * D + 8 * c);
            const uint2 w = *p;
            *p = make_uint2(rescale_e4m3x4(w.x, f_old), rescale_e4m3x4(w.y, f_old));
        } else if (!TURNED && a.clear) {
            *reinterpret_cast<uint2*>(cache + pos * D + 8 * c) = make_uint2(0u, 0u);
        }
    }
    if constexpr (TURNED) {
        __syncthreads();
        // four tokens of a column at a time; words that hold older or no tokens too are merged
        for (int u = tid; u < D * BT / 4; u += kThreads) {
            const int d = u / (BT / 4), p = u % (BT / 4) * 4;
            uint32_t* out = reinterpret_cast<uint32_t*>(cache + d * BT + p);
            const uint32_t w = *reinterpret_cast<const uint32_t*>(lds + d * (BT + 4) + p);
            if (p >= t0 && p + 4 <= t1) {
                *out = w;
            } else if (p >= t1) {
                if (a.clear) *out = 0;
            } else if (p + 4 > t0 || grown) {
                const uint32_t old = *out, moved = grown ? rescale_e4m3x4(old, f_old) : old;
                uint32_t r = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t from = p + j < t0 ? moved : p + j < t1 ? w : a.clear ? 0u : old;
                    r |= from & (255u << 8 * j);
                }
                *out = r;
            }
        }
    }
}

template <class T, int DK, int DV, int BT>
__global__ void __launch_bounds__(kThreads) attn_append_kernel(AttnAppendArgs a) {
    __shared__ __attribute__((aligned(16))) char lds[DV * (BT + 4)];
    __shared__ float wave_max[4];
    const int head = blockIdx.x % a.Hk;
    const AppendBlock b = find_block(a, blockIdx.x / a.Hk, threadIdx.x & 63);
    if (b.seq < 0 || b.block >= a.max_blocks) return;
    const int page = a.table[static_cast<int64_t>(b.seq) * a.max_blocks + b.block];
    if (page < 0 || page >= a.num_blocks) return;
    if (blockIdx.y == 0)
        append_page<T, DK, BT, false>(a, b, page, head, lds, wave_max);
    else
        append_page<T, DV, BT, true>(a, b, page, head, lds, wave_max);
}

template <class T, int DK, int DV>
hipError_t append_dims(const AttnAppendArgs& a, hipStream_t stream) {
    // blocks written into: at most one per new token, and two partial ones per sequence
    const int64_t most = static_cast<int64_t>(a.total) / a.bt + 2ll * a.N;
    const dim3 grid(static_cast<unsigned>((most < a.total ? most : a.total) * a.Hk), 2);
    switch (a.bt) {
        case 16: attn_append_kernel<T, DK, DV, 16><<<grid, kThreads, 0, stream>>>(a); break;
        case 32: attn_append_kernel<T, DK, DV, 32><<<grid, kThreads, 0, stream>>>(a); break;
        case 64: attn_append_kernel<T, DK, DV, 64><<<grid, kThreads, 0, stream>>>(a); break;
        default: attn_append_kernel<T, DK, DV, 128><<<grid, kThreads, 0, stream>>>(a); break;
    }
    return hipGetLastError();
}

template <class T>
hipError_t append_type(const AttnAppendArgs& a, int dk, int dv, hipStream_t stream) {
    if (dk == 64) return dv == 64 ? append_dims<T, 64, 64>(a, stream) : append_dims<T, 64, 128>(a, stream);
    return dv == 64 ? append_dims<T, 128, 64>(a, stream) : append_dims<T, 128, 128>(a, stream);
}

// ---------------------------------------------------------------------------
// Decode.  Rows are the T query tokens of a sequence times the heads of one kv head, 16 to a tile;
// a wave takes 64 keys a step:
//   S^T = K Q^T       A = K (bytes to bf16, exact), B = Q; four 16x16 tiles of keys
//   O^T += V^T P^T    A = V^T from the turned cache, B = P as S^T's accumulators hold it
// Tile row i of tile t is key 16 (i / 4) + 4 t + i % 4, so that lane group g (= lane / 16) ends up
// with the weights of keys 16 g .. 16 g + 15, which are one 16-byte load of V^T per column.  Every
// byte of the cache goes from memory to registers once, 16 at a time, without LDS.  A step of a wave
// is 16 KiB; two waves a SIMD keep 128 KiB a compute unit asked for.  Bound by memory: 64 contexts
// of up to 16000 (1.0 GB) 185 us and the join, 5.4 TB/s, four of 8192 to 131072 with 4 tokens each
// 116 us, 5.4 TB/s; a plain read of 1 GiB reaches 6.2.  (168 registers, three waves a SIMD, spill:
// 280 us for the first.)
// ---------------------------------------------------------------------------
template <class T>
struct Parts {  // of bf16 that hold a query or weight of this type
    static constexpr int n = T::bytes == 2 ? 1 : 3;
};

__device__ __forceinline__ bf16x8 e4m3_to_bf16(uint32_t lo, uint32_t hi) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
    const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// x[8] as N bf16 vectors whose sum is x up to 2^-8N.
template <int N>
__device__ __forceinline__ void split_bf16(const float (&x)[8], bf16x8 (&out)[N]) {
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(r[2 * j], r[2 * j + 1]);
        out[n] = __builtin_bit_cast(bf16x8, w);
        if (n + 1 < N)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t half = w[j >> 1];
                r[j] -= __uint_as_float(j & 1 ? half & 0xffff0000u : half << 16);
            }
    }
}

// How the batch is cut, the same in every workgroup: all sequences into pieces of `steps` steps, a
// size that makes about a.pieces of them per kv head in all, whatever the lengths.
struct DecodePlan {
    const AttnDecodeArgs& a;
    int lane, steps;

    __device__ __forceinline__ int context(int n) const {
        return min(max(a.context_len[n], 0), a.max_blocks * a.bt);  // host-checked: below 2^31
    }
    __device__ __forceinline__ int steps_of(int n) const {
        return n < a.N ? (context(n) + kStepKeys - 1) / kStepKeys : 0;
    }
    __device__ __forceinline__ DecodePlan(const AttnDecodeArgs& args, int l) : a(args), lane(l), steps(0) {
        if (a.pieces == 0) return;  // not cut
        int all = 0;
        for (int n = 0; n < a.N; n += kWave) all += wave_total(steps_of(n + lane));
        steps = decode_piece_steps(all, a.pieces, decode_table_steps(a.max_blocks, a.bt));
    }
    __device__ __forceinline__ int pieces_of(int n) const { return (steps_of(n) + steps - 1) / steps; }
    // Sequence and place in it of piece t; sequence -1 past the last.
    __device__ __forceinline__ int2 find(int t) const {
        for (int n = 0; n < a.N; n += kWave) {
            const int2 at = find_in(pieces_of(n + lane), t);
            if (at.x >= 0) return make_int2(n + at.x, at.y);
            t = at.y;
        }
        return make_int2(-1, 0);
    }
    // Pieces of the sequences before n.
    __device__ __forceinline__ int before(int n) const {
        int sum = 0;
        for (int m = 0; m < n; m += kWave) sum += wave_total(m + lane < n ? pieces_of(m + lane) : 0);
        return sum;
    }
};

template <class T, int DK, int DV, int RT>
__global__ void __launch_bounds__(kThreads, RT == 1 ? 2 : 1) attn_decode_kernel(AttnDecodeArgs a) {
    constexpr int NP = Parts<T>::n;
    constexpr int kRowsT = 16 * RT, kLd = DV + 4;  // floats between rows of the exchange
    __shared__ __attribute__((aligned(16))) float part[4][kRowsT][kLd];
    __shared__ float part_m[4][kRowsT], part_l[4][kRowsT];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int per = a.Hk * a.row_groups, piece = blockIdx.x / per, rest = blockIdx.x % per;
    // (row groups of one kv head are Hk workgroups apart: with Hk a multiple of 8, in one XCD's L2)
    const int kvh = rest % a.Hk, row0 = rest / a.Hk * kRowsT;
    const int G = a.H / a.Hk, R = a.T * G;
    const DecodePlan plan(a, lane);
    const int2 at = a.pieces ? plan.find(piece) : make_int2(piece, 0);
    const int n = __builtin_amdgcn_readfirstlane(at.x);
    if (n < 0) return;
    const int ctx = plan.context(n), keys = a.pieces ? plan.steps * kStepKeys : ctx;
    const int begin = __builtin_amdgcn_readfirstlane(at.y) * keys, end = min(ctx - begin, keys) + begin;
    const bool whole = ctx <= keys;  // the sequence's only piece: its output is final

    bf16x8 qf[RT][DK / 32][NP];
    int see[RT];  // last key that the lane's row sees
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int row = min(row0 + 16 * rt + i, R - 1), t = row / G;
        see[rt] = ctx - a.T + t;
        const int64_t at = (static_cast<int64_t>(n) * a.T + t) * a.ldq + (kvh * G + row % G) * DK;
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) {
            const int64_t d = at + 64 * (s >> 1) + 16 * g + 8 * (s & 1);
            const float4 lo = load4<T>(a.q, d), hi = load4<T>(a.q, d + 4);
            const float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            split_bf16<NP>(x, qf[rt][s]);
        }
    }
    f32x4 acc[RT][DV / 16];
    float m[RT], mc[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = -INFINITY, mc[rt] = 0.f, l[rt] = 0.f;
#pragma unroll
        for (int d = 0; d < DV / 16; ++d) acc[rt][d] = f32x4{};
    }

    const int32_t* table = a.table + static_cast<int64_t>(n) * a.max_blocks;
    // page of the 16 keys from key on, or -1 (past the end, absent, out of range)
    auto page_of = [&](int key) {
        const int p = table[min(key >> a.bt_log2, a.max_blocks - 1)];
        return key < end && p >= 0 && p < a.num_blocks ? p : -1;
    };
    u32x4 kb[4][DK / 64], vb[DV / 16];
    float ks, vs;
    auto load_k = [&](int base, int page) {  // page: of quarter i / 4
        const int64_t head = static_cast<int64_t>(max(page, 0)) * a.Hk + kvh;
        const int64_t row = head * a.bt + ((base + 16 * (i >> 2)) & (a.bt - 1));
        const uint8_t* p = a.k_cache + (row + (i & 3)) * DK + 16 * g;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int x = 0; x < DK / 64; ++x)
                kb[t][x] = *reinterpret_cast<const u32x4*>(p + 4 * t * DK + 64 * x);
    };
    auto load_v = [&](int base, int page) {  // page: of quarter g
        const int64_t head = static_cast<int64_t>(max(page, 0)) * a.Hk + kvh;
        const uint8_t* p = a.v_cache + (head * DV + i) * a.bt + ((base + 16 * g) & (a.bt - 1));
#pragma unroll
        for (int d = 0; d < DV / 16; ++d) vb[d] = *reinterpret_cast<const u32x4*>(p + 16 * d * a.bt);
    };
    auto load_scales = [&](int page) {
        const int64_t head = static_cast<int64_t>(max(page, 0)) * a.Hk + kvh;
        ks = a.k_scale[head], vs = a.v_scale[head];
    };

    // Pages are looked up two steps ahead: loads come back in order, so one looked up in the step
    // that uses it would wait for the values asked for before.  The last step, which asks for
    // nothing, is a copy of its own: behind a branch inside the step, the compiler would wait for
    // every load at the step's end.
    int base = begin + 64 * wave;
    int page_now = page_of(base + 16 * g), page_k = page_of(base + 16 * (i >> 2));
    int page_v = page_of(base + kStepKeys + 16 * g);
    if (base < end) {
        load_k(base, page_k);
        load_scales(page_now);
        load_v(base, page_now);
    }
    page_k = page_of(base + kStepKeys + 16 * (i >> 2));
    const auto step = [&](auto MORE) __attribute__((always_inline)) {
        constexpr bool more = decltype(MORE)::value;
        const int next = base + kStepKeys;
        int page_k2 = -1, page_v2 = -1;
        if constexpr (more)
            page_k2 = page_of(next + kStepKeys + 16 * (i >> 2)), page_v2 = page_of(next + kStepKeys + 16 * g);
        __builtin_amdgcn_sched_barrier(0);  // loads stay where they are: moved, they would take copies
        f32x4 s[RT][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) s[rt][t] = f32x4{};
#pragma unroll
            for (int x = 0; x < DK / 32; ++x) {
                const u32x4 b = kb[t][x >> 1];
                const bf16x8 kf = x & 1 ? e4m3_to_bf16(b[2], b[3]) : e4m3_to_bf16(b[0], b[1]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
                        s[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[rt][x][p], s[rt][t], 0, 0, 0);
            }
        }
        float ks_now = ks, vs_now = vs;
        asm volatile("" : "+v"(ks_now), "+v"(vs_now));  // taken here, not at the end of the step before
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (more) {
            load_k(next, page_k);
            load_scales(page_v);
        }
        __builtin_amdgcn_sched_barrier(0);
        // an absent page's scale is another page's: its keys get the weight 0 times 0
        const float c = a.scale * kLog2e * ks_now, vscale = page_now < 0 ? 0.f : vs_now;
        // (both sides are formed: no branch stands between the products and the first use of s)
        const bool edge = (base + 64 > ctx - a.T + 1) | (__any(page_now < 0) != 0);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[rt][t][j] *= c;
            if (edge) {
                const int last = page_now < 0 ? -1 : see[rt] - (base + 16 * g);
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (4 * t + j > last) s[rt][t][j] = -INFINITY;
            }
            float mx = s[rt][0][0];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) mx = fmaxf(mx, s[rt][t][j]);
            mx = fmaxf(mx, __shfl_xor(mx, 16, kWave));
            mx = fmaxf(mx, __shfl_xor(mx, 32, kWave));
            if (__any(mx > mc[rt] + 8.f || (m[rt] == -INFINITY && mx > m[rt]))) {
                const float mn = fmaxf(m[rt], mx);
                const float al = m[rt] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[rt] - mn);
                m[rt] = mn;
                mc[rt] = mn == -INFINITY ? 0.f : mn;
                l[rt] *= al;
#pragma unroll
                for (int d = 0; d < DV / 16; ++d)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[rt][d][j] *= al;
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = __builtin_amdgcn_exp2f(s[rt][t][j] - mc[rt]);
                    l[rt] += p;
                    s[rt][t][j] = p * vscale;
                }
        }
        if (edge) {  // what no row sees may be anything: as zeros it stays out of the products
            const int live = page_now < 0 ? 0 : min(max(end - (base + 16 * g), 0), 16);
#pragma unroll
            for (int d = 0; d < DV / 16; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int keep = live - 4 * j;
                    vb[d][j] &= keep >= 4 ? 0xffffffffu : keep <= 0 ? 0u : (1u << 8 * keep) - 1u;
                }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            bf16x8 pf[RT][NP];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const f32x4 x = s[rt][2 * u], y = s[rt][2 * u + 1];
                const float p[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
                split_bf16<NP>(p, pf[rt]);
            }
#pragma unroll
            for (int d = 0; d < DV / 16; ++d) {
                const bf16x8 vf = e4m3_to_bf16(vb[d][2 * u], vb[d][2 * u + 1]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
                        acc[rt][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[rt][p], acc[rt][d], 0, 0, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (more) {
            load_v(next, page_v);
            page_now = page_v, page_v = page_v2, page_k = page_k2;
            base = next;
        }
    };
    if (base < end) {
        while (base + kStepKeys < end) step(std::true_type{});
        step(std::false_type{});
    }

    // the four waves' parts of a row come together
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        l[rt] += __shfl_xor(l[rt], 16, kWave);
        l[rt] += __shfl_xor(l[rt], 32, kWave);
        if (g == 0) part_m[wave][16 * rt + i] = m[rt], part_l[wave][16 * rt + i] = l[rt];
#pragma unroll
        for (int d = 0; d < DV / 16; ++d)
            *reinterpret_cast<f32x4*>(&part[wave][16 * rt + i][16 * d + 4 * g]) = acc[rt][d];
    }
    __syncthreads();
    for (int u = tid; u < kRowsT * (DV / 4); u += kThreads) {
        const int row = u / (DV / 4), d = u % (DV / 4) * 4;
        if (row0 + row >= R) break;
        float M = -INFINITY;
#pragma unroll
        for (int v = 0; v < 4; ++v) M = fmaxf(M, part_m[v][row]);
        float L = 0.f;
        f32x4 o = f32x4{};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float mv = part_m[v][row], f = mv == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mv - M);
            L = fmaf(f, part_l[v][row], L);
            const f32x4 x = *reinterpret_cast<const f32x4*>(&part[v][row][d]);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = fmaf(f, x[j], o[j]);
        }
        const int t = (row0 + row) / G, head = kvh * G + (row0 + row) % G;
        if (whole) {
            const int64_t out = (static_cast<int64_t>(n) * a.T + t) * a.H + head;
            const float inv = L == 0.f ? 0.f : 1.f / L;
            store4<T>(a.o, out * DV + d, make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv));
        } else {
            const int64_t p = (static_cast<int64_t>(piece) * a.T + t) * a.H + head;
            *reinterpret_cast<f32x4*>(a.part_o + p * DV + d) = o;
            if (d == 0) a.part_ml[p] = make_float2(M, L);
        }
    }
}

// Joins a row's pieces, a wave a row; 64 pieces at a time, lane i with the maximum and sum of the
// i-th.
template <class T, int DV>
__global__ void __launch_bounds__(kThreads) attn_combine_kernel(AttnDecodeArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rows = a.T * a.H;
    if (row >= static_cast<int64_t>(a.N) * rows) return;
    const int n = static_cast<int>(row) / rows, in = static_cast<int>(row) % rows;  // host-checked: 2^22 rows
    const DecodePlan plan(a, lane);
    const int pieces = __builtin_amdgcn_readfirstlane(plan.pieces_of(n));
    if (pieces == 1) return;  // written by its workgroup
    const int64_t first = plan.before(n);
    constexpr int kLanes = DV / 4, kSide = kWave / kLanes;  // lanes of a row, pieces side by side
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < pieces; base += kWave) {
        const int here = min(pieces - base, kWave);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < here) ml = a.part_ml[(first + base + lane) * rows + in];
        float m = fmaxf(ml.x, M);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
        const float f = ml.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - m);
        const float old = M == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(M - m);
        M = m;
        L = fmaf(L, old, wave_sum(f * ml.y));
        o = f4_mul(o, old);
        // two or four pieces a load instruction, eight of those in flight
        const float* p = a.part_o + ((first + base) * rows + in) * DV + 4 * (lane % kLanes);
        for (int s0 = 0; s0 < here; s0 += 8 * kSide) {
            float4 x[8];
            float w[8];
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int at = s0 + s * kSide + lane / kLanes;
                x[s] = load4<F32>(p, static_cast<int64_t>(min(at, here - 1)) * rows * DV);
                w[s] = __shfl(f, at & (kWave - 1), kWave);
                w[s] = at < here ? w[s] : 0.f;
            }
#pragma unroll
            for (int s = 0; s < 8; ++s) o = f4_scale_fma(w[s], x[s], o);
        }
    }
#pragma unroll
    for (int d = kLanes; d < kWave; d *= 2) o = f4_add(o, f4_shfl_xor(o, d));
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if (lane < kLanes) store4<T>(a.o, row * DV + 4 * lane, f4_mul(o, inv));
}

// Row tiles of a workgroup.  More rows than a workgroup's go to further groups, which find the cache
// in the L2: up to 32 rows as one or two groups of 16 (24 rows, 8 x 8000 keys: 39 us; one group
// of 32, at half the waves a compute unit, 48), more as groups of 32 (64 rows, 4 x 60000 keys:
// 173 us; groups of 16 215, one of 64 230).
int row_tiles(int T, int H, int Hk) { return T * (H / Hk) <= 32 ? 1 : 2; }

template <class T, int DK, int DV, int RT>
hipError_t decode_rows(const AttnDecodeArgs& a, hipStream_t stream) {
    const int64_t wgs = (a.pieces ? attn_decode_most_pieces(a.N, a.pieces) : a.N) * a.Hk * a.row_groups;
    attn_decode_kernel<T, DK, DV, RT><<<dim3(static_cast<unsigned>(wgs)), kThreads, 0, stream>>>(a);
    if (a.pieces) {
        const int64_t rows = static_cast<int64_t>(a.N) * a.T * a.H;
        attn_combine_kernel<T, DV><<<dim3(static_cast<unsigned>((rows + 3) / 4)), kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <class T, int DK, int DV>
hipError_t decode_dims(const AttnDecodeArgs& a, hipStream_t stream) {
    return row_tiles(a.T, a.H, a.Hk) == 1 ? decode_rows<T, DK, DV, 1>(a, stream)
                                          : decode_rows<T, DK, DV, 2>(a, stream);
}

template <class T>
hipError_t decode_type(const AttnDecodeArgs& a, int dk, int dv, hipStream_t stream) {
    if (dk == 64) return dv == 64 ? decode_dims<T, 64, 64>(a, stream) : decode_dims<T, 64, 128>(a, stream);
    return dv == 64 ? decode_dims<T, 128, 64>(a, stream) : decode_dims<T, 128, 128>(a, stream);
}

}  // namespace

hipError_t launch_attn_append(const AttnAppendArgs& a, int bf16, int dk, int dv, hipStream_t stream) {
    return bf16 ? append_type<BF16>(a, dk, dv, stream) : append_type<F32>(a, dk, dv, stream);
}

int attn_decode_row_groups(int T, int H, int Hk) {
    const int rows = 16 * row_tiles(T, H, Hk);
    return (T * (H / Hk) + rows - 1) / rows;
}

int attn_decode_pieces(int N, int T, int H, int Hk, int bt, int max_blocks) {
    const int64_t per = static_cast<int64_t>(Hk) * attn_decode_row_groups(T, H, Hk);
    return decode_pieces(N, per, decode_table_steps(max_blocks, bt));
}

int64_t attn_decode_most_pieces(int N, int pieces) { return static_cast<int64_t>(pieces) + N; }

hipError_t launch_attn_decode(const AttnDecodeArgs& a, int bf16, int dk, int dv, hipStream_t stream) {
    return bf16 ? decode_type<BF16>(a, dk, dv, stream) : decode_type<F32>(a, dk, dv, stream);
}

}  // namespace kda
