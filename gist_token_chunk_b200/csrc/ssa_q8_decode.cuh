// ssa_q8_decode.cuh -- the decode step over the 8-bit cache, three kernels on the
// caller's stream by programmatic dependent launch:
//
//   score   x[m, t, h] = (q_h . code[m, t]) / sqrt(d) for every gist and head, kept,
//           and s[m] = ks[m] * max over h and t, as an order-preserving key;
//   select  the k = min(topk, M_b) largest keys, ties to the lower chunk;
//   attend  one online softmax per head over the unselected gists (their kept
//           logits and values), the selected chunks' raw rows and the tail, split
//           over CTAs, joined by the last CTA of each (sequence, KV head).
//
// Bound by HBM: (M g + (M - k) g + 2 k C + 2 T) d bytes per (sequence, KV head). Heads go
// in groups of eight, and above G = 8 everything but the gist keys is read once a group.
// Kept logits are 16 bytes a gist (G <= 4; to 8 heads 32, above 64), written and read, in
// place of a second read of its d bytes of key.
// One block scale multiplies whole rows, so it never touches the codes: the
// keys' scale multiplies the logit, the values' scale the softmax weight.
// The codes become f16 (exact) in registers, on the way to m16n8k16.  Its
// fragments take any order of the contracted index, so a lane's 16-byte piece of a
// key row is its fragment:
//   Q K^T   contraction step s of lane t uses bytes 4 s .. 4 s + 3 of the lane's 16.
//           Heads fill 8 of the 16 rows of A; an fp32 query is the sum of two f16
//           numbers (22 bits), the second in rows 8-15.
//   P V     weights likewise as high and low part (22 bits); column i of lane g is
//           byte i of the d / 8 that the lane reads.
// The halves of an accumulator are added at the end, so the second parts cost no
// instruction.  The same steps on e4m3 itself (m16n8k32, queries as sums of 4-bit
// pieces) are as exact, but on this device they run as conversions and f16 steps,
// of the queries too, each time: the scores then issued 343 instructions for 16 rows.
//
// Measured (B200, us a step in a CUDA graph; in brackets the bytes at the copy's
// rate): 32K batch 24.2 (6.4), 128K 26.3 (6.5), 512K 32.6 (10.2), 32 sequences with
// d = 128 82.6 (41.6).  The first three are bound by the latencies of three dependent
// kernels; the last by the attention's instructions a tile and its CTAs' start and end.
#pragma once

#include "ssa_q8.h"
#include "ssa_q8_cache.cuh"

namespace ssa_q8 {

constexpr int kHeads = 8;          // heads of one accumulator
constexpr int kTile = 16;          // context rows a warp takes at a time
constexpr int kWarps = 4;          // warps of an attend CTA
constexpr int kScoreWarps = 4;
// Gist rows of a score CTA (at least one chunk).  256, 512, 1024: 24.9, 24.2, 26.4 us a
// step on the 32K batch, 26.3, 26.3, 28.1 on 128K, 84.4, 82.6, 84.4 on 32 sequences.
constexpr int kScoreRows = 512;
constexpr int kSelThreads = 512;
constexpr int kSelectKeys = 16;    // keys of a thread that bisects
constexpr int kMaxTopk = 1024;
constexpr int kMaxSplits = 1024;   // splits of one (sequence, KV head, head group)
constexpr int kMinTiles = 8;       // raw tiles of a split, as long as there are splits enough
// A softmax weight times its value scale enters f16 over a power of two that its head
// raises when such a product passes kWeightMax: the largest is then put at 2^7 to 2^9, and
// the next raise is a factor of 2^6 away.  So f16's least step, 2^-24, is under 2^-31 of
// the largest product so far, half of it the most that a weight loses, whatever other
// blocks' scales are (scales under 2^-100 count as that).
constexpr float kWeightUp = 8.0f;  // log2
constexpr float kWeightMax = 32768.0f, kSumMax = 1152921504606846976.0f;  // 2^15, 2^60
// What a tile counts for in a split's share.  4, 5, 6, 8 to 8: 27.0, 26.3, 26.4, 27.6 us
// (128K batch), 95.7, 82.6, 83.7, 84.9 (32 sequences).
constexpr int kGistWeight = 5, kRawWeight = 8;
// A warp's ring: copies in flight, and the stage in use.  2, 3, 4: 32.1, 32.6, 43.1 us
// (512K batch; four leave room for fewer CTAs), 87.3, 82.6, 81.9 (32 sequences).
constexpr int kStages = 3;
template <int D>
constexpr int kGroup = 128 / D;    // tiles of a stage
// A partial result of one head: o[D], held over 2^(y + x), then y, x, and the sum, held
// over 2^x.  y stays apart: past 2^24 a logit's 32 bits do not hold x + y.  In shared memory the D / 8 columns that a lane holds
// lie 4 words further apart, and so do the records: stores of 16 bytes then share no
// bank.
template <int D>
constexpr int kRecord = D + 4;
template <int D>
constexpr int kColumns = D / 8 + 4;
template <int D>
constexpr int kJoin = 8 * kColumns<D> + 4;

struct DecodeArgs {
    int B, Hkv, Hq, G, NG;  // NG: groups of 8 heads
    int n_max, M_max, C, g, topk;
    int LG;                 // heads of a kept logit row: 4 or 8
    int nch;                // chunks of a score CTA
    int tpc;                // tiles of a raw chunk
    FastDiv by_g, by_tpc;
    const void* q;
    const uint8_t *k_raw, *v_raw, *k_gist, *v_gist;
    const float *k_raw_s, *v_raw_s, *k_gist_s, *v_gist_s;
    const int32_t* seq_lens;
    float* out;
    int32_t* sel;
    uint32_t* keys;  // [B * Hkv, key_stride]
    int key_stride;
    float* logits;   // [NG, B * Hkv, M_max * g, LG], log2, without the key's scale
    int* done;       // [B * Hkv * NG] CTAs of the attention that are through
    float* part;     // [attend grid, 8, d + 4]
    float qk_scale;  // log2(e) / sqrt(d)
    int smem_mask, smem_sel;  // byte offsets in the attend CTA's shared memory
};

// ------------------------------------------------------------- fragments ---

// The queries of one head group as f16 fragments.  Lane (g = lane / 4, t = lane % 4)
// holds head g's elements 64 h + 16 t + [0, 16).  The head is scaled by a power of
// two so that its largest element lies in [2^13, 2^14): a bf16 query is then exact
// (elements 2^28 times smaller than the largest lose bits), an fp32 one the sum of
// two parts.  One warp makes them for the CTA; they lie in shared memory, a 16-byte
// word a lane, and are read back where they are used.
template <class E, int D>
struct QueryFrag {
    static constexpr int NP = sizeof(E) == 2 ? 1 : 2;  // parts
    struct Shared {
        uint4 w[NP][D / 32][32];  // [part][32 dims][lane]: 8 elements
        float scale[kHeads];      // of the sums, to logits in log2; NaN: no such head
    };
    const Shared* sm;

    // By one warp: the A operand's rows (the B operand's columns) of its 8 heads.
    struct Raw {
        uint4 v[D * sizeof(E) / 64];
    };
    static __device__ __forceinline__ void fetch(Raw& r, const E* q, bool valid) {
        constexpr int N = sizeof(E);  // 16-byte words of 16 elements
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int i = 0; i < N; ++i)
                r.v[N * h + i] = ldg128_if(q + 64 * h + 16 * (threadIdx.x & 3) + 16 / N * i, valid);
    }
    static __device__ __forceinline__ void make(Shared* sm, const Raw& raw, bool valid,
                                                float qk_scale) {
        const int lane = threadIdx.x & 31;
        float x[D / 4];
        const int t = threadIdx.x & 3;
#pragma unroll
        for (int i = 0; i < D * (int)sizeof(E) / 64; ++i) {
            const uint32_t v[4] = {raw.v[i].x, raw.v[i].y, raw.v[i].z, raw.v[i].w};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if constexpr (sizeof(E) == 2) {
                    x[8 * i + 2 * n] = __uint_as_float(v[n] << 16);
                    x[8 * i + 2 * n + 1] = __uint_as_float(v[n] & 0xffff0000u);
                } else {
                    x[4 * i + n] = __uint_as_float(v[n]);
                }
            }
        }
        uint32_t top = 0u;  // the largest magnitude's bits, of the finite elements
#pragma unroll
        for (int i = 0; i < D / 4; ++i) {
            const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
            top = max(top, u < 0x7f800000u ? u : 0u);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = top ? max((int)(top >> 23) - 127 - 13, -100) : 0;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        if (t == 0)
            sm->scale[lane >> 2] = valid ? __uint_as_float((uint32_t)(127 + e) << 23) * qk_scale
                                         : __uint_as_float(0x7fffffffu);
#pragma unroll
        for (int h = 0; h < D / 32; ++h) {
            uint32_t w[NP][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[8 * h + 2 * i] * down, b = x[8 * h + 2 * i + 1] * down;
                w[0][i] = pack_f16(a, b);
                if constexpr (NP == 2) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[0][i]));
                    // (an infinite element is all in the first part)
                    w[1][i] = pack_f16(isinf(a) ? 0.0f : a - f.x, isinf(b) ? 0.0f : b - f.y);
                }
            }
#pragma unroll
            for (int p = 0; p < NP; ++p)
                sm->w[p][h][lane] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
        }
    }

    // Heads x 8 key rows: x[e] is head lane / 4, row 2 (lane % 4) + e.  k: the lane's
    // bytes of row lane / 4.
    __device__ __forceinline__ void dot(float (&x)[2], const uint4 (&k)[D / 64]) const {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < D / 32; ++h) {
            const uint4 a = sm->w[0][h][threadIdx.x & 31];
            uint4 c = make_uint4(0, 0, 0, 0);
            if constexpr (NP == 2) c = sm->w[1][h][threadIdx.x & 31];
            uint32_t b[4];
            e4m3x4_to_f16(h & 1 ? k[h / 2].z : k[h / 2].x, b[0], b[1]);
            e4m3x4_to_f16(h & 1 ? k[h / 2].w : k[h / 2].y, b[2], b[3]);
            mma_f16(s, a.x, c.x, a.y, c.y, b[0], b[1]);
            mma_f16(s, a.z, c.z, a.w, c.w, b[2], b[3]);
        }
        x[0] = NP == 2 ? s[0] + s[2] : s[0];
        x[1] = NP == 2 ? s[1] + s[3] : s[1];
    }

    // 16 key rows x heads: x[2 i + e] is row lane / 4 + 8 i, head 2 (lane % 4) + e;
    // the queries are the 8-column operand.  k[i]: the lane's bytes of row lane / 4 + 8 i.
    __device__ __forceinline__ void dot16(float (&x)[4], const uint4 (&k)[2][D / 64]) const {
        x[0] = x[1] = x[2] = x[3] = 0.0f;
#pragma unroll
        for (int h = 0; h < D / 32; ++h) {
            uint32_t a[8];  // [row half][contraction pair]
            e4m3x4_to_f16(h & 1 ? k[0][h / 2].z : k[0][h / 2].x, a[0], a[1]);
            e4m3x4_to_f16(h & 1 ? k[0][h / 2].w : k[0][h / 2].y, a[2], a[3]);
            e4m3x4_to_f16(h & 1 ? k[1][h / 2].z : k[1][h / 2].x, a[4], a[5]);
            e4m3x4_to_f16(h & 1 ? k[1][h / 2].w : k[1][h / 2].y, a[6], a[7]);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const uint4 b = sm->w[p][h][threadIdx.x & 31];
                mma_f16(x, a[0], a[4], a[1], a[5], b.x, b.y);
                mma_f16(x, a[2], a[6], a[3], a[7], b.z, b.w);
            }
        }
    }
};

// 16 bytes (4: a scale) to shared memory, without waiting.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copy16_or_zero(void* dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_end_group() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A length outside [1, n_max] counts as a sequence without context.
__device__ __forceinline__ int valid_len(const DecodeArgs& a, int b) {
    const int n = a.seq_lens[b];
    return n >= 1 && n <= a.n_max ? n : 0;
}

// ----------------------------------------------------------------- score ---

// One CTA of 4 warps takes nch consecutive chunks of one (sequence, KV head); a
// warp takes 64 (d = 128: 32) gist rows at a time, 16 to a matrix step with the
// keys as the 16-row operand.  The first loads go out before the length is
// known (they stay inside the pair's M_max chunks).  With g a multiple of 8 the
// eight rows of a half step belong to one chunk, and one warp-wide maximum
// covers them and all heads; otherwise each row's maximum goes to shared memory.
// The loads in flight live in registers and L1, not in shared memory: so the scores
// read at 0.97 of the copy's rate (32 sequences, d = 128).
template <class E, int D, int NG>
__global__ void __launch_bounds__(128, D == 64 && sizeof(E) == 2 && NG == 1 ? 6 : 4)
    score_kernel(DecodeArgs a) {
    // In this order: the later kernels read inputs before their own wait, so they may
    // start only once the work before this step is through.
    wait_prerequisites();
    launch_dependents();
    extern __shared__ uint32_t best[];  // [nch], then the chunks' scales
    __shared__ typename QueryFrag<E, D>::Shared query[NG];
    const int tiles = (a.M_max + a.nch - 1) / a.nch;
    const int pair = blockIdx.x / tiles;
    const int m0 = (blockIdx.x % tiles) * a.nch;
    const int b = pair / a.Hkv, j = pair % a.Hkv;
    if (m0 == 0 && threadIdx.x < a.NG) a.done[pair * a.NG + threadIdx.x] = 0;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gid = lane >> 2, t = lane & 3;
    const uint8_t* base = a.k_gist + ((long long)pair * a.M_max + m0) * a.g * D;
    constexpr int U = D == 64 ? 4 : 2;  // 16-row steps in flight
    uint4 k[U][2][D / 64];
    auto load = [&](int r, int rows) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = r + 16 * u + 8 * i + gid;
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    k[u][i][h] = ldg128_if(base + (long long)row * D + 64 * h + 16 * t, row < rows);
            }
    };
    // the queries first: behind all keys' loads they would arrive last
    const int M = valid_len(a, b) / a.C;
    const int h = 8 * warp + gid;
    const bool ok = warp < NG && h < a.G;
    typename QueryFrag<E, D>::Raw raw;
    QueryFrag<E, D>::fetch(
        raw, static_cast<const E*>(a.q) + ((long long)b * a.Hq + j * a.G + (ok ? h : 0)) * D, ok);
    int r = warp * 16 * U;
    const int most = min(a.nch, a.M_max - m0);
    load(r, most * a.g);
    float* scale = reinterpret_cast<float*>(best + a.nch);
    for (int i = threadIdx.x; i < most; i += 128) {
        best[i] = 0u;
        copy4(scale + i, a.k_gist_s + (long long)pair * a.M_max + m0 + i);
    }
    copies_end_group();
    if (warp < NG) QueryFrag<E, D>::make(&query[warp], raw, ok, a.qk_scale);
    const int m1 = min(M, m0 + a.nch);
    if (m0 >= m1) {
        copies_wait<0>();
        return;
    }
    const int rows = (m1 - m0) * a.g;
    __syncthreads();
    float sc[NG][2];  // scales of heads 2t, 2t + 1: no maximum takes the NaN of an absent head
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        sc[n][0] = query[n].scale[2 * t];
        sc[n][1] = query[n].scale[2 * t + 1];
    }
    const bool whole = (a.g & 7) == 0;
    float* keep = a.logits + ((long long)pair * a.M_max + m0) * a.g * a.LG + 2 * t;
    for (; r < rows; r += kScoreWarps * 16 * U) {
        float x[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u][0] = x[u][1] = -INFINITY;
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                float s[4];
                QueryFrag<E, D>{&query[n]}.dot16(s, k[u]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 y = make_float2(s[2 * i] * sc[n][0], s[2 * i + 1] * sc[n][1]);
                    x[u][i] = fmaxf(x[u][i], fmaxf(y.x, y.y));
                    const int row = r + 16 * u + 8 * i + gid;
                    if (row < rows && 2 * t < a.LG)
                        __stcg(reinterpret_cast<float2*>(
                                   keep + ((long long)n * gridDim.x / tiles * a.M_max * a.g + row) * a.LG),
                               y);
                }
            }
        }
        const int at = r;
        if (r + kScoreWarps * 16 * U < rows) load(r + kScoreWarps * 16 * U, rows);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = at + 16 * u + 8 * i;
                uint32_t key = score_key(x[u][i]);
                if (whole) {
                    key = __reduce_max_sync(0xffffffffu, key);
                    if (lane == 0 && row < rows) atomicMax(&best[a.by_g.div(row)], key);
                } else {
                    key = max(key, __shfl_xor_sync(0xffffffffu, key, 1));
                    key = max(key, __shfl_xor_sync(0xffffffffu, key, 2));
                    if (t == 0 && row + gid < rows) atomicMax(&best[a.by_g.div(row + gid)], key);
                }
            }
    }
    copies_wait<0>();
    __syncthreads();
    for (int i = threadIdx.x; i < m1 - m0; i += 128)
        a.keys[(long long)pair * a.key_stride + m0 + i] = score_key(key_score(best[i]) * scale[i]);
}

// ---------------------------------------------------------------- select ---

// Exclusive sum over the CTA's kSelThreads threads; sh: a word a warp.  Every
// thread passes one barrier; the caller puts one before sh is written again.
__device__ __forceinline__ int scan_before(int x, int* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int run = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
    }
    if (lane == 31) sh[warp] = run;
    __syncthreads();
    return run - x + __reduce_add_sync(0xffffffffu, lane < warp ? sh[lane] : 0);
}

// Up to 512 chunks a warp, their keys in registers: bisection of the key that
// exactly k keys reach (k < M).  It ends early where a gap between the k-th and the
// next key is met, after about log2 M steps on scores without ties, and after 32 at
// the k-th key itself where keys tie; of those the first are taken.  A step is one
// count: no barrier with one warp, one with more.  (Against histograms and ranks:
// 28.8 -> 28.0 us a step on the 128K batch, 36.9 -> 35.0 on 512K.  The CTA runs its code
// once, from cold instruction caches, so short code counts.)
__device__ __forceinline__ void select_bisect(const uint32_t* keys, int M, int k, int32_t* sel,
                                              int* sh) {
    constexpr int K = kSelectKeys;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
    const int m0 = warp * 32 * K + lane;
    uint32_t key[K], low = 0xffffffffu, high = 0u;
#pragma unroll
    for (int i = 0; i < K; ++i) key[i] = __ldcg(keys + min(m0 + 32 * i, M - 1));
#pragma unroll
    for (int i = 0; i < K; ++i) {
        if (m0 + 32 * i >= M) key[i] = 0u;  // no score has key 0
        high = max(high, key[i]);
        low = min(low, key[i] - 1u);
    }
    int turn = 0;
    // sum over the CTA; two sets of words, so one barrier a call
    auto all = [&](int x) {
        x = __reduce_add_sync(0xffffffffu, x);
        if (W > 1) {
            int* at = sh + 16 * (turn++ & 1);
            if (lane == 0) at[warp] = x;
            __syncthreads();
            x = __reduce_add_sync(0xffffffffu, lane < W ? at[lane] : 0);
        }
        return x;
    };
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (W > 1) {
        uint32_t* at = reinterpret_cast<uint32_t*>(sh) + 32;
        if (lane == 0) {
            at[warp] = low;
            at[16 + warp] = high;
        }
        __syncthreads();
        low = __reduce_min_sync(0xffffffffu, at[lane < W ? lane : 0]);
        high = __reduce_max_sync(0xffffffffu, at[16 + (lane < W ? lane : 0)]);
    }
    // all M keys reach low, none high; at least k reach low throughout
    ++low;
    ++high;
    bool exact = false;
    while (!exact && high - low > 1u) {
        const uint32_t mid = low + (high - low) / 2u;
        int c = 0;
#pragma unroll
        for (int i = 0; i < K; ++i) c += key[i] >= mid;
        c = all(c);
        exact = c == k;
        if (c >= k)
            low = mid;
        else
            high = mid;
    }
    // Keys from `above` on, and the first of those that equal low where it ties: lane i
    // takes the word of chunks 32 i .. 32 i + 31.
    const uint32_t above = exact ? low : high;
    uint32_t v = 0u, e = 0u;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const uint32_t x = __ballot_sync(0xffffffffu, key[i] >= above);
        const uint32_t y = __ballot_sync(0xffffffffu, key[i] == low);
        if (lane == i) {
            v = x;
            e = exact ? 0u : y;
        }
    }
    // exclusive sums over the words before: selected, equal
    auto sum_before = [&](int x) {
        int run = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += y;
        }
        int first = 0;
        if (W > 1) {
            int* at = sh + 16 * (turn++ & 1);
            if (lane == 31) at[warp] = run;
            __syncthreads();
            first = __reduce_add_sync(0xffffffffu, lane < warp ? at[lane] : 0);
        }
        return first + run - x;
    };
    if (!exact) {
        const int need = k - all(__popc(v));
        int take = min(need - sum_before(__popc(e)), __popc(e));
        for (; take > 0; --take) {  // its lowest bits
            v |= e & (0u - e);
            e &= e - 1u;
        }
    }
    for (int at = sum_before(__popc(v)); v; v &= v - 1u)
        sel[at++] = warp * 32 * K + 32 * lane + __ffs(v) - 1;
}

// More chunks than that: radix select of the k-th largest, 11 + 11 + 10 bits, then an
// ordered compaction; each thread owns consecutive chunks and reads their keys from L2.
__device__ __noinline__ void select_radix(const uint32_t* keys, int M, int k, int32_t* sel, int* hist,
                                          int* sh) {
    constexpr int T = kSelThreads, PER = 2048 / T;
    const int tid = threadIdx.x;
    const int E = (M + T - 1) / T;
    const int lo = min(M, tid * E), hi = min(M, lo + E);
    uint32_t prefix = 0, mask = 0;
    int need = k;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
        __syncthreads();
        for (int i = tid; i < 2048; i += T) hist[i] = 0;
        __syncthreads();
        for (int m = lo; m < hi; ++m) {
            const uint32_t key = __ldcg(keys + m);
            if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & digits], 1);
        }
        __syncthreads();
        // thread t holds bins 2047 - PER t downwards
        int sum = 0;
        for (int i = 0; i < PER; ++i) sum += hist[2047 - PER * tid - i];
        int at = scan_before(sum, sh);
        if (at < need && at + sum >= need) {
            int b = 2047 - PER * tid;
            while (at + hist[b] < need) at += hist[b--];
            sh[32] = b;
            sh[33] = need - at;
            sh[34] = hist[b];
        }
        __syncthreads();
        prefix |= (uint32_t)sh[32] << shift;
        mask |= digits << shift;
        need = sh[33];
        if (sh[34] == need) break;  // every key of the digit is wanted
    }
    // keys above the prefix, and the first `need` that equal it
    int above = 0, equal = 0;
    for (int m = lo; m < hi; ++m) {
        const uint32_t v = __ldcg(keys + m) & mask;
        above += v > prefix;
        equal += v == prefix;
    }
    __syncthreads();
    int pa = scan_before(above, sh);
    __syncthreads();
    int pe = scan_before(equal, sh);
    for (int m = lo; m < hi; ++m) {
        const uint32_t v = __ldcg(keys + m) & mask;
        if (v > prefix) {
            sel[pa + min(pe, need)] = m;
            ++pa;
        } else if (v == prefix) {
            if (pe < need) sel[pa + pe] = m;
            ++pe;
        }
    }
}

// One CTA a (sequence, KV head), of a warp for every 512 chunks (at most kSelThreads).
__global__ void __launch_bounds__(kSelThreads) select_kernel(DecodeArgs a) {
    launch_dependents();
    __shared__ int sh[64];
    extern __shared__ int hist[];  // 2048, with kSelThreads
    const int pair = blockIdx.x, b = pair / a.Hkv;
    const int M = valid_len(a, b) / a.C;
    const int k = min(a.topk, M);
    int32_t* sel = a.sel + (long long)pair * a.topk;
    wait_prerequisites();
    for (int i = k + threadIdx.x; i < a.topk; i += blockDim.x) sel[i] = -1;
    if (k == M) {
        for (int i = threadIdx.x; i < k; i += blockDim.x) sel[i] = i;
        return;
    }
    const uint32_t* keys = a.keys + (long long)pair * a.key_stride;
    if (M <= kSelectKeys * (int)blockDim.x)
        select_bisect(keys, M, k, sel, sh);
    else
        select_radix(keys, M, k, sel, hist, sh);
}

// ---------------------------------------------------------------- attend ---

// Tiles of one (sequence, KV head): gist rows, then the selected chunks' rows and
// the tail's (tpc tiles a chunk; the tail is the last chunk, and shorter).
struct Counts {
    int M, k, T, gist, raw;
    // A split's share goes by bytes: a raw tile reads keys and values, a gist tile
    // values and logits.
    __device__ __forceinline__ int weight() const { return kGistWeight * gist + kRawWeight * raw; }
    __device__ __forceinline__ int tile_at(int w) const {
        const int g = kGistWeight * gist;
        return w < g ? (w + kGistWeight - 1) / kGistWeight : gist + (w - g + kRawWeight - 1) / kRawWeight;
    }
};
__device__ __forceinline__ Counts counts_of(const DecodeArgs& a, int n) {
    Counts c;
    c.M = n / a.C;
    c.T = n - c.M * a.C;
    c.k = min(a.topk, c.M);
    c.gist = (c.M * a.g + kTile - 1) / kTile;
    c.raw = c.k * a.tpc + (c.T + kTile - 1) / kTile;
    return c;
}

// What a warp's stage holds: P tiles of 16 rows, keys (gists: logits, [row][LG]),
// values, and their scales.  Row r of a tile, r = t + 4 e + 8 i, is column 2 t + e of
// the matrix steps' half i, so
//   keys    lie in slot 2 t + e of the half (slot g is lane g's row),
//   scales  in word 4 t + e + 2 i (a lane reads its four rows' at once),
// and 16-byte pieces are swizzled so that no two lanes of a phase share a bank.
template <int D>
struct Stage {
    static constexpr int P = kGroup<D>;
    alignas(16) uint8_t k[P][kTile * D];
    uint8_t v[P][kTile * D];
    float ks[P][kTile], vs[P][kTile];
    int rows[P];  // that exist
    int pad[4 - P];

    static __device__ __forceinline__ int k_at(int r, int piece) {
        const int slot = (r & 8) + 2 * (r & 3) + ((r >> 2) & 1);
        return slot * D + 16 * (D == 64 ? piece : piece ^ 4 * (slot & 1));
    }
    static __device__ __forceinline__ int v_at(int r, int piece) {
        return r * D + 16 * (piece ^ (D == 64 ? (r & 2) : 2 * (r & 3)));
    }
    static __device__ __forceinline__ int scale_at(int r) {
        return 4 * (r & 3) + ((r >> 2) & 1) + 2 * (r >> 3);
    }
};

// CTAs of one attend kernel that are resident on an SM.
template <int D>
constexpr int kResident = D == 64 ? 4 : 3;

template <class E, int D>
__global__ void __launch_bounds__(32 * kWarps, kResident<D>) attend_kernel(DecodeArgs a, int* status) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int plan[4];
    __shared__ typename QueryFrag<E, D>::Shared query;
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem + a.smem_mask);
    int* sel = reinterpret_cast<int*>(smem + a.smem_sel);
    Stage<D>* ring = reinterpret_cast<Stage<D>*>(smem) + (threadIdx.x >> 5) * kStages;
    float* merge = reinterpret_cast<float*>(smem);  // when the rings are through
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gid = lane >> 2, t = lane & 3;
    const int units = a.Hkv * a.NG;  // independent rows of splits of one sequence

    // Plan: every sequence gets ceil(weight / quota) splits for each of its
    // units.  With quota >= all weights / (grid - units) the splits fit the grid,
    // whatever the lengths.
    if (warp == 0) {
        const int mine = lane < a.B ? counts_of(a, valid_len(a, lane)).weight() : 0;
        long long all = mine;
        int longest = mine;
        for (int b = lane + 32; b < a.B; b += 32) {
            const int c = counts_of(a, valid_len(a, b)).weight();
            all += c;
            longest = max(longest, c);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        longest = __reduce_max_sync(0xffffffffu, longest);
        const int room = (int)gridDim.x - a.B * units;
        int quota = room > 0 ? (int)min(ceil((double)all * units / room), (double)longest) : longest;
        quota = max(quota, max(kMinTiles * kRawWeight, (longest + kMaxSplits - 1) / kMaxSplits));
        if (lane == 0) plan[0] = -1;
        __syncwarp();
        int first = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            const int c = b0 == 0 ? mine : b < a.B ? counts_of(a, valid_len(a, b)).weight() : 0;
            const int s = b < a.B ? max(1, (c + quota - 1) / quota) : 0;
            int run = s * units;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            const int at = (int)blockIdx.x - (first + run - s * units);
            if (at >= 0 && at < s * units) {
                plan[0] = b;
                plan[1] = at / s;  // unit
                plan[2] = at % s;  // split
                plan[3] = s;
            }
            first += __shfl_sync(0xffffffffu, run, 31);
        }
    }
    __syncthreads();
    const int b = plan[0];
    if (b < 0) {
        wait_prerequisites();
        return;
    }
    const int unit = plan[1], split = plan[2], ns = plan[3];
    const int j = unit / a.NG, ng = unit % a.NG;
    const long long pair = (long long)b * a.Hkv + j;
    const int n = valid_len(a, b);
    const int heads = min(kHeads, a.G - ng * kHeads);
    float* out = a.out + ((long long)b * a.Hq + (long long)j * a.G + ng * kHeads) * D;
    if (n == 0) {
        wait_prerequisites();
        for (int i = tid; i < heads * D; i += 32 * kWarps) out[i] = 0.0f;
        if (tid == 0) atomicCAS(status, 0, (int)SSA_ERR_DEVICE_STATUS);
        return;
    }
    const Counts c = counts_of(a, n);
    const int share = c.weight() / ns, more = c.weight() % ns;
    const int w0 = split * share + min(split, more);
    const int u0 = c.tile_at(w0), u1 = c.tile_at(w0 + share + (split < more));

    if (warp == kWarps - 1) {
        typename QueryFrag<E, D>::Raw raw;
        QueryFrag<E, D>::fetch(raw,
                               static_cast<const E*>(a.q) +
                                   ((long long)b * a.Hq + (long long)j * a.G + ng * kHeads +
                                    (gid < heads ? gid : 0)) * D,
                               gid < heads);
        QueryFrag<E, D>::make(&query, raw, gid < heads, a.qk_scale);
    }
    const QueryFrag<E, D> q{&query};

    // the selection, and a bitmap of the selected chunks among this split's gist rows
    const int g0 = u0 < c.gist ? (int)a.by_g.div(u0 * kTile) : 0;  // first chunk of its gist rows
    const int g1 = u0 < c.gist
                       ? (int)a.by_g.div(min(min(u1, c.gist) * kTile, c.M * a.g) - 1) + 1
                       : 0;
    for (int i = tid; i < (g1 - g0 + 31) / 32; i += 32 * kWarps) mask[i] = 0u;

    // Copies of the tiles u .. u + P - 1 into a stage: everything but the gists'
    // logits (early), those (late), or both.  Gists of selected chunks come along:
    // their addresses do not wait for the selection.  Rows that do not exist are
    // zeros, logits of such rows anything.  A tile's rows are contiguous: piece i of
    // lane l is its 16 bytes 16 l + 512 i.
    constexpr int P = kGroup<D>, PIECES = D / 16, STEP = 32 / PIECES;
    const int Mg = c.M * a.g, rr = lane & 15;
    const float* lg = a.logits + (((long long)ng * a.B * a.Hkv + pair) * a.M_max * a.g) * a.LG + 4 * lane;
    const uint8_t* vg = a.v_gist + pair * a.M_max * a.g * D + 16 * lane;
    const uint8_t* kr = a.k_raw + pair * a.n_max * D + 16 * lane;
    const uint8_t* vr = a.v_raw + pair * a.n_max * D + 16 * lane;
    const float* sg = (lane < 16 ? a.k_gist_s : a.v_gist_s) + pair * a.M_max;
    const float* sr = (lane < 16 ? a.k_raw_s : a.v_raw_s) + pair * a.M_max;
    int k_to[kTile / STEP];  // places in the stage; v: one more 512 bytes on for each i
    const int v_to = Stage<D>::v_at(lane / PIECES, lane % PIECES);
#pragma unroll
    for (int i = 0; i < kTile / STEP; ++i) k_to[i] = Stage<D>::k_at(i * STEP + lane / PIECES, lane % PIECES);
    auto fetch_logits = [&](Stage<D>& s, int u) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (u + p < min(u1, c.gist) && lane < 4 * a.LG)
                copy16(s.k[p] + 16 * lane, lg + (long long)(u + p) * (kTile * a.LG));
    };
    auto fetch = [&](Stage<D>& s, int u) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (u + p >= u1) break;
            int rows, m;
            const float* sc;
            const uint8_t *kp = nullptr, *vp;
            if (u + p < c.gist) {
                const int r0 = (u + p) * kTile;
                rows = Mg - r0;
                m = (int)a.by_g.div(min(r0 + rr, Mg - 1));
                sc = sg;
                vp = vg + (long long)(u + p) * (kTile * D);
            } else {
                const int x = u + p - c.gist, i = (int)a.by_tpc.div(x), r0 = (x - i * a.tpc) * kTile;
                m = sel[i];
                rows = (i < c.k ? a.C : c.T) - r0;
                sc = sr;
                const long long at = ((long long)m * a.C + r0) * D;
                kp = kr + at;
                vp = vr + at;
            }
            if (rows >= kTile) {
#pragma unroll
                for (int i = 0; i < kTile / STEP; ++i) copy16(s.v[p] + v_to + 512 * i, vp + 512 * i);
                if (kp) {
#pragma unroll
                    for (int i = 0; i < kTile / STEP; ++i) copy16(s.k[p] + k_to[i], kp + 512 * i);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < kTile / STEP; ++i) {
                    const int r = i * STEP + lane / PIECES;
                    const bool in = r < rows;
                    copy16_or_zero(s.v[p] + v_to + 512 * i, in ? vp + 512 * i : vg, in);
                    if (kp)
                        copy16_or_zero(s.k[p] + Stage<D>::k_at(r, lane % PIECES), in ? kp + 512 * i : vg, in);
                }
            }
            copy4((lane < 16 ? s.ks[p] : s.vs[p]) + Stage<D>::scale_at(rr), sc + m);
            if (lane == 0) s.rows[p] = rows;
        }
    };

    // A warp takes P tiles at a time, every fourth such group, and fetches kStages - 1
    // groups ahead; the values of groups of gists alone do not wait for the selection.
    const int first = u0 + P * warp;
    int ahead = 0;
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i)
        if (ahead == i && min(first + i * P * kWarps + P, u1) <= c.gist) {
            fetch(ring[i], first + i * P * kWarps);
            ++ahead;
        }
    wait_prerequisites();
    __syncthreads();
    bool met = false;
    for (int i = tid; i <= c.k; i += 32 * kWarps) {
        const int m = i < c.k ? __ldcg(a.sel + pair * a.topk + i) : c.M;  // the last: the tail
        sel[i] = m;
        if (m >= g0 && m < g1) {
            atomicOr(&mask[(m - g0) >> 5], 1u << ((m - g0) & 31));
            met = true;
        }
    }
    met = __syncthreads_or(met);  // some of this split's gists are a selected chunk's
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
        if (i >= ahead) fetch(ring[i], first + i * P * kWarps);
        fetch_logits(ring[i], first + i * P * kWarps);
        copies_end_group();
    }

    const bool here = gid < heads;
    const float qs = here ? query.scale[gid] : 0.0f;
    // The sum l of the weights p = 2^(x - m), and acc, the sum of p * scale * 2^(kWeightUp - k) *
    // code. m and k are whole numbers. m is the maximum of the logits (log2) when it was last
    // set; k is that of x - m + log2(scale), which m alone does not tell: the head may attend to
    // blocks whose scales are far under others'.
    float m = -INFINITY, k = -INFINITY, up = 0.0f, l = 0.0f;
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    int slot = 0;
    for (int u = first; u < u1; u += P * kWarps) {
        copies_wait<kStages - 2>();
        __syncwarp();  // every lane's copies; and the stage used last is free
        Stage<D>& free = ring[slot == 0 ? kStages - 1 : slot - 1];
        fetch(free, u + (kStages - 1) * P * kWarps);
        fetch_logits(free, u + (kStages - 1) * P * kWarps);
        copies_end_group();
        const Stage<D>& s = ring[slot];
        slot = slot == kStages - 1 ? 0 : slot + 1;

        float x[P][4], vs[P][4];  // [tile][2 i + e]
        uint32_t see[P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (u + p < c.gist) {
                // absent heads read another's
                const float* y = reinterpret_cast<const float*>(s.k[p]) + t * a.LG + (gid & (a.LG - 1));
#pragma unroll
                for (int i = 0; i < 4; ++i) x[p][i] = y[4 * i * a.LG];
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 k[D / 64];
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        k[h] = *reinterpret_cast<const uint4*>(
                            s.k[p] + (8 * i + gid) * D + 16 * (D == 64 ? t : (4 * h + t) ^ 4 * (gid & 1)));
                    float y[2];
                    q.dot(y, k);
                    x[p][2 * i] = y[0] * qs;
                    x[p][2 * i + 1] = y[1] * qs;
                }
            }
            const float4 ks = *reinterpret_cast<const float4*>(s.ks[p] + 4 * t);
            const float4 sv = *reinterpret_cast<const float4*>(s.vs[p] + 4 * t);
            x[p][0] *= ks.x;
            x[p][1] *= ks.y;
            x[p][2] *= ks.z;
            x[p][3] *= ks.w;
            vs[p][0] = sv.x;
            vs[p][1] = sv.y;
            vs[p][2] = sv.z;
            vs[p][3] = sv.w;
            // rows that exist and are not a selected chunk's gists
            const int rows = u + p < u1 ? s.rows[p] : 0;
            see[p] = rows >= kTile ? 0xffffu : (1u << rows) - 1u;
            if (met && u + p < c.gist) {
                const int i = (int)a.by_g.div(min((u + p) * kTile + rr, Mg - 1)) - g0;
                see[p] &= ~__ballot_sync(0xffffffffu, (mask[i >> 5] >> (i & 31)) & 1u);
            }
            if (see[p] != 0xffffu) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!((see[p] >> (t + 4 * i)) & 1u)) {
                        x[p][i] = -INFINITY;
                        vs[p][i] = 0.0f;
                    }
            }
        }
        float w[P][4], sum, most;
        auto weigh = [&](float ref) {
            sum = 0.0f;
            most = 0.0f;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float y = ex2(x[p][i] - ref);
                    sum += y;
                    w[p][i] = y * vs[p][i] * up;
                    most = fmaxf(most, w[p][i]);
                }
        };
        // with the references so far; the first tile finds none, and a NaN shows in the sum
        weigh(m);
        if (__any_sync(0xffffffffu, here && !(most <= kWeightMax && l + sum <= kSumMax))) {
            float tx = -INFINITY, ty = -INFINITY;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) tx = fmaxf(tx, x[p][i]);
            tx = fmaxf(tx, __shfl_xor_sync(0xffffffffu, tx, 1));
            tx = fmaxf(tx, __shfl_xor_sync(0xffffffffu, tx, 2));
            const float nx = fmaxf(m, ceilf(tx)), ref = nx == -INFINITY ? 0.0f : nx;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = (int)(__float_as_uint(vs[p][i]) >> 23 & 255u) - 127;
                    ty = fmaxf(ty, x[p][i] - ref + (float)max(e, kMinScaleExp));
                }
            ty = fmaxf(ty, __shfl_xor_sync(0xffffffffu, ty, 1));
            ty = fmaxf(ty, __shfl_xor_sync(0xffffffffu, ty, 2));
            // over the new m, acc's reference is `old`; what it holds is kept if that is the largest
            const float old = m == -INFINITY ? -INFINITY : k + (m - nx);
            const float nk = fmaxf(old, ceilf(ty));
            const float f = nk == -INFINITY ? 0.0f : pow2(old - nk);
            l *= pow2(m - nx);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                acc[i][0] *= f;
                acc[i][1] *= f;
                acc[i][2] *= f;
                acc[i][3] *= f;
            }
            m = nx;
            k = nk;
            up = nk == -INFINITY ? 0.0f : pow2(kWeightUp - nk);
            weigh(ref);
        }
        l += sum;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                hi[i] = pack_f16(w[p][2 * i], w[p][2 * i + 1]);
                const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi[i]));
                lo[i] = pack_f16(w[p][2 * i] - back.x, w[p][2 * i + 1] - back.y);
            }
            // the lane's D / 8 columns of rows t + 4 e + 8 i
            uint32_t v[2][2][D / 32];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = t + 4 * e + 8 * i;
                    if constexpr (D == 64) {
                        const uint2 w = *reinterpret_cast<const uint2*>(
                            s.v[p] + Stage<D>::v_at(r, gid >> 1) + 8 * (gid & 1));
                        v[i][e][0] = w.x;
                        v[i][e][1] = w.y;
                    } else {
                        const uint4 w =
                            *reinterpret_cast<const uint4*>(s.v[p] + Stage<D>::v_at(r, gid));
                        v[i][e][0] = w.x;
                        v[i][e][1] = w.y;
                        v[i][e][2] = w.z;
                        v[i][e][3] = w.w;
                    }
                }
            if (see[p] != 0xffffu) {  // a NaN in a masked row would pass its zero weight
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (!((see[p] >> (t + 4 * e + 8 * i)) & 1u)) {
#pragma unroll
                            for (int w = 0; w < D / 32; ++w) v[i][e][w] = 0u;
                        }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                // bytes of the four rows, by column
                uint32_t b0[4], b1[4];
                e4m3x4_to_f16(__byte_perm(v[0][0][w], v[0][1][w], 0x5140), b0[0], b0[1]);
                e4m3x4_to_f16(__byte_perm(v[0][0][w], v[0][1][w], 0x7362), b0[2], b0[3]);
                e4m3x4_to_f16(__byte_perm(v[1][0][w], v[1][1][w], 0x5140), b1[0], b1[1]);
                e4m3x4_to_f16(__byte_perm(v[1][0][w], v[1][1][w], 0x7362), b1[2], b1[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_f16(acc[4 * w + i], hi[0], lo[0], hi[1], lo[1], b0[i], b1[i]);
            }
        }
    }
    copies_wait<0>();
    __syncthreads();  // the rings become the merge area

    // join the warps in shared memory
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    constexpr int W = kRecord<D>, J = kJoin<D>, CS = kColumns<D>;
    float* mine = merge + (warp * kHeads + gid) * J;
#pragma unroll
    for (int i = 0; i < D / 8; i += 4)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(mine + (2 * t + e) * CS + i) =
                make_float4(acc[i][e] + acc[i][2 + e], acc[i + 1][e] + acc[i + 1][2 + e],
                            acc[i + 2][e] + acc[i + 2][2 + e], acc[i + 3][e] + acc[i + 3][2 + e]);
    if (t == 0)
        *reinterpret_cast<float4*>(mine + 8 * CS) = make_float4(k, m, l, 0.0f);
    __syncthreads();
    float* part = a.part + (long long)blockIdx.x * kHeads * W;
    for (int i = 4 * tid; i < heads * D; i += 4 * 32 * kWarps) {
        const int h = i / D, x = i % D;
        float ty = -INFINITY, tx = -INFINITY;
        float4 r[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            r[w] = *reinterpret_cast<const float4*>(merge + (w * kHeads + h) * J + 8 * CS);
            tx = fmaxf(tx, r[w].y);
        }
        const float rx = tx == -INFINITY ? 0.0f : tx;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            r[w].x += r[w].y - rx;
            ty = fmaxf(ty, r[w].x);
        }
        const float ry = ty == -INFINITY ? 0.0f : ty;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = pow2(r[w].x - ry);
            const float4 y = *reinterpret_cast<const float4*>(merge + (w * kHeads + h) * J +
                                                              x / (D / 8) * CS + x % (D / 8));
            o.x += f * y.x;
            o.y += f * y.y;
            o.z += f * y.z;
            o.w += f * y.w;
            sum += pow2(r[w].y - rx) * r[w].z;
        }
        if (ns == 1) {
            const float r = 1.0f / sum, f = pow2(ry - kWeightUp);  // apart: both may be small
            out[i] = o.x * r * f;
            out[i + 1] = o.y * r * f;
            out[i + 2] = o.z * r * f;
            out[i + 3] = o.w * r * f;
        } else {
            __stcg(reinterpret_cast<float4*>(part + h * W + x), o);
            if (x == 0)
                __stcg(reinterpret_cast<float4*>(part + h * W + D), make_float4(ty, tx, sum, 0.0f));
        }
    }
    if (ns == 1) return;

    // the last split of the unit joins them all, in the order of the splits
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        plan[3] = atomicAdd(a.done + pair * a.NG + ng, 1);
        __threadfence();
    }
    __syncthreads();
    if (plan[3] != ns - 1) return;
    // A warp takes a head: lane s the references and sum of split s (and s + 32, ...),
    // then D / 32 columns of every split's o.
    const float* all = part - (long long)split * kHeads * W;
    float* weight = merge + warp * ns;  // the merge area holds 4 * ns
    for (int h = warp; h < heads; h += kWarps) {
        const float* rec = all + h * W;
        constexpr int V = D / 32, N = D == 64 ? 16 : 8;  // columns of a lane; splits at a time
        float r[N][V];
        auto fetch_some = [&](int s0) {
#pragma unroll
            for (int s = 0; s < N; ++s)
                if (s0 + s < ns) {
                    const float* p = rec + (long long)(s0 + s) * kHeads * W + V * lane;
                    if constexpr (V == 2) {
                        const float2 f = __ldcg(reinterpret_cast<const float2*>(p));
                        r[s][0] = f.x;
                        r[s][1] = f.y;
                    } else {
                        const float4 f = __ldcg(reinterpret_cast<const float4*>(p));
                        r[s][0] = f.x;
                        r[s][1] = f.y;
                        r[s][2] = f.z;
                        r[s][3] = f.w;
                    }
                }
        };
        fetch_some(0);
        auto refs = [&](int s) {
            return __ldcg(reinterpret_cast<const float4*>(rec + (long long)s * kHeads * W + D));
        };
        const float4 f0 = refs(min(lane, ns - 1));  // most units have no more splits than that
        float ty = -INFINITY, tx = f0.y, sum = 0.0f;
        for (int s = lane + 32; s < ns; s += 32) tx = fmaxf(tx, refs(s).y);
#pragma unroll
        for (int o = 16; o; o >>= 1) tx = fmaxf(tx, __shfl_xor_sync(0xffffffffu, tx, o));
        const float rx = tx == -INFINITY ? 0.0f : tx;
        for (int s = lane; s < ns; s += 32) {
            const float4 f = s == lane ? f0 : refs(s);
            const float y = f.x + (f.y - rx);
            weight[s] = y;
            ty = fmaxf(ty, y);
            sum += f.z * pow2(f.y - rx);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            ty = fmaxf(ty, __shfl_xor_sync(0xffffffffu, ty, o));
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        const float ry = ty == -INFINITY ? 0.0f : ty;
        __syncwarp();
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.0f;
        for (int s0 = 0; s0 < ns; s0 += N) {
#pragma unroll
            for (int s = 0; s < N; ++s)
                if (s0 + s < ns) {
                    const float f = pow2(weight[s0 + s] - ry);
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] += f * r[s][i];
                }
            if (s0 + N < ns) fetch_some(s0 + N);
        }
        const float f = pow2(ry - kWeightUp);
#pragma unroll
        for (int i = 0; i < V; ++i) out[h * D + V * lane + i] = o[i] / sum * f;
        __syncwarp();
    }
}

}  // namespace ssa_q8
