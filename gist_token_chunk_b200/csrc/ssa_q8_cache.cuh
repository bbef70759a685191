// ssa_q8_cache.cuh -- writing the 8-bit cache and reading it back.
//
// A cache tensor holds N rows of d e4m3 codes per (sequence, KV head), in
// blocks of R consecutive rows with one fp32 scale each: value = code * scale.
// The scale is a power of two, the smallest s >= 2^-100 with amax / s <= 448.
// A power of two costs e4m3 nothing (its relative step is the same at every
// magnitude), x / s is exact, and when a later append finds a larger row in a
// block, the block's earlier rows move to the new scale without another
// rounding, except where they fall below the smallest normal code.
//
// Both kernels are bound by HBM: the append reads e and writes 1 byte an
// element, the read back the other way round (33.7 us for 2 x 32K tokens; 128K
// tokens back in 62.1 us, 0.99 of the copy's rate).
#pragma once

#include "ssa_q8.h"

namespace ssa_q8 {

constexpr int kMinScaleExp = -100;

struct AppendArgs {
    const void* x[2];         // new rows of keys, values
    long long xs[2][3];       // strides in elements: sequence, head, row
    uint8_t* code[2];         // [B, Hkv, N, d]
    float* scale[2];          // [B, Hkv, N / R]
    const int32_t* start;     // [B]
    const int32_t* count;     // [B] or NULL: T
    int B, Hkv, T, R, nblk;   // nblk: blocks a sequence can touch
    int N;
    int tensors;              // 1 or 2
    uint32_t items;
    FastDiv by_heads, by_blocks, by_rows;
};

// 8 consecutive elements of a row
template <class E>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = ldg128(p); }
    __device__ __forceinline__ void load_if(const __nv_bfloat16* p, bool in) { v = ldg128_if(p, in); }
    // running maximum of the magnitudes, as bits; an infinity or NaN is larger
    // than every number.  Two lanes of 16 bits, joined by peak_value.
    __device__ __forceinline__ uint32_t peak(uint32_t m) const {
        m = __vmaxu2(m, v.x & 0x7fff7fffu);
        m = __vmaxu2(m, v.y & 0x7fff7fffu);
        m = __vmaxu2(m, v.z & 0x7fff7fffu);
        return __vmaxu2(m, v.w & 0x7fff7fffu);
    }
    static __device__ __forceinline__ float peak_value(uint32_t m) {
        return __uint_as_float(max(m << 16, m & 0xffff0000u));
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Vec8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = ldg128(p);
        b = ldg128(p + 4);
    }
    __device__ __forceinline__ void load_if(const float* p, bool in) {
        a = ldg128_if(p, in);
        b = ldg128_if(p + 4, in);
    }
    __device__ __forceinline__ uint32_t peak(uint32_t m) const {
        m = max(max(m, a.x & 0x7fffffffu), max(a.y & 0x7fffffffu, a.z & 0x7fffffffu));
        m = max(max(m, a.w & 0x7fffffffu), max(b.x & 0x7fffffffu, b.y & 0x7fffffffu));
        return max(m, max(b.z & 0x7fffffffu, b.w & 0x7fffffffu));
    }
    static __device__ __forceinline__ float peak_value(uint32_t m) { return __uint_as_float(m); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
};

// The rows [lo, hi) of block blk that a span of `count` rows from `start` holds;
// false: none. In 64 bits until the block is known to hold some: a grid for T rows
// has blocks past a shorter span's end, and near the largest N those start past 2^31.
__host__ __device__ __forceinline__ bool rows_in_block(int start, int count, long long blk, int R,
                                                       int& lo, int& hi) {
    const long long b0 = blk * R, end = (long long)start + count;
    if (b0 >= end || b0 + R <= start) return false;
    lo = (int)(b0 > start ? b0 : start);
    hi = (int)(b0 + R < end ? b0 + R : end);
    return lo < hi;
}

__device__ __forceinline__ bool finite_bits(float x) {
    return (__float_as_uint(x) & 0x7fffffffu) < 0x7f800000u;
}

// Smallest power of two s >= 2^-100 with amax / s <= 448 = 1.75 * 2^8
// (amax = m * 2^e with 1 <= m < 2: s = 2^(e - 8) while m <= 1.75, else one up).
__device__ __forceinline__ float pow2_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    k = max(k, kMinScaleExp);
    return __uint_as_float((uint32_t)(k + 127) << 23);
}

// Codes of 8 values divided by the scale (inv = 1 / scale).  e4m3 has no
// infinity: one becomes NaN rather than the largest number (the conversion keeps a
// NaN but saturates an infinity, so blocks that hold one take `checked`).
__device__ __forceinline__ uint2 quantise8(float (&f)[8], float inv, bool checked) {
    if (checked) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!finite_bits(f[i])) f[i] = __uint_as_float(0x7fffffffu);
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = f32x2_to_e4m3(f[2 * i] * inv, f[2 * i + 1] * inv);
    return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
}

// GROUP threads own one (tensor, sequence, head, block): the block's amax is
// known only after its last row, so up to KEEP vectors a thread stay in
// registers between the two passes; rows beyond them are read a second time.
// A warp owns a block while its new rows fit 32 * KEEP vectors (no barrier,
// four blocks a CTA), larger ones take 64, 128 or 256 threads.  Half as many vectors
// a thread, on more threads, took twice as long: the work per thread then no longer
// covers its start.  33.7 us for 2 x 32K tokens, 0.91 of the copy's rate.
template <class E>
constexpr int kAppendKeep = sizeof(E) == 2 ? 16 : 8;
template <class E, int D, int GROUP>
__global__ void __launch_bounds__(GROUP == 32 ? 128 : GROUP) append_kernel(AppendArgs a, int* status) {
    constexpr int KEEP = kAppendKeep<E>;
    constexpr int VR = D / 8;  // vectors in a row
    constexpr int PER = GROUP == 32 ? 4 : 1;
    __shared__ uint32_t red[8];
    const int tid = threadIdx.x % GROUP;
    const uint32_t item = blockIdx.x * PER + threadIdx.x / GROUP;
    if (item >= a.items) return;
    // tensors and heads fastest: a token's rows of all heads, which lie side by side
    // in a projection's output, are read at about the same time
    const int kv = a.tensors == 2 ? item & 1 : 0;
    const uint32_t bjx = a.tensors == 2 ? item >> 1 : item, bx = a.by_heads.div(bjx);
    const int j = (int)(bjx - bx * a.Hkv);
    const int b = (int)a.by_blocks.div(bx);
    const int blk_i = (int)(bx - (uint32_t)b * a.nblk);

    wait_prerequisites();
    const int start = a.start[b];
    const int count = a.count ? a.count[b] : a.T;
    if (count == 0) return;
    if (start < 0 || count < 0 || count > a.T || start > a.N - count) {
        if (tid == 0) atomicCAS(status, 0, (int)SSA_ERR_DEVICE_STATUS);
        return;
    }
    const long long blk = (long long)a.by_rows.div(start) + blk_i;
    const long long b0 = blk * a.R;  // first row of the block
    int lo, hi;                      // its new rows
    if (!rows_in_block(start, count, blk, a.R, lo, hi)) return;
    const int nv = (hi - lo) * VR;
    const long long rs = a.xs[kv][2];
    // vector tid of the new rows, and its place; vector tid + i GROUP is i steps on
    constexpr int STEP = GROUP / VR;
    const E* src = static_cast<const E*>(a.x[kv]) + b * a.xs[kv][0] + j * a.xs[kv][1] +
                   (lo - start + tid / VR) * rs + tid % VR * 8;
    uint8_t* code = a.code[kv] + ((long long)b * a.Hkv + j) * a.N * D;
    uint8_t* dst = code + (long long)lo * D + tid * 8;
    float* sp = a.scale[kv] + ((long long)b * a.Hkv + j) * (a.N / a.R) + blk;

    const float old = lo > b0 ? *sp : 0.0f;  // earlier rows: their scale
    Vec8<E> keep[KEEP];
    uint32_t peak = 0u;
    const bool full = nv >= KEEP * GROUP;  // every thread holds KEEP vectors: no tests
    if (full) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) keep[i].load(src + i * STEP * rs);
    } else {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) keep[i].load_if(src + i * STEP * rs, tid + i * GROUP < nv);
    }
#pragma unroll
    for (int i = 0; i < KEEP; ++i) peak = keep[i].peak(peak);
#pragma unroll 1
    for (int i = KEEP; tid + i * GROUP < nv; ++i) {
        Vec8<E> r;
        r.load(src + i * STEP * rs);
        peak = r.peak(peak);
    }
    auto join = [&](uint32_t m) {  // over the group
        m = __reduce_max_sync(0xffffffffu, m);
        if (GROUP > 32) {
            __syncthreads();  // every thread of the CTA has the same item
            if ((tid & 31) == 0) red[tid >> 5] = m;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < GROUP / 32; ++i) m = max(m, red[i]);
        }
        return m;
    };
    // magnitudes order like their bits
    uint32_t top = join(__float_as_uint(Vec8<E>::peak_value(peak)));
    const bool checked = top >= 0x7f800000u;  // some are not finite: over the others
    if (checked) {
        uint32_t m = 0u;
#pragma unroll 1
        for (int i = 0; tid + i * GROUP < nv; ++i) {
            Vec8<E> r;
            r.load(src + i * STEP * rs);
            float f[8];
            r.get(f);
#pragma unroll
            for (int n = 0; n < 8; ++n)
                if (finite_bits(f[n])) m = max(m, __float_as_uint(f[n]) & 0x7fffffffu);
        }
        top = join(m);
    }
    const float s = fmaxf(pow2_scale(__uint_as_float(top)), old);
    const float inv = 1.0f / s;
    auto put = [&](const Vec8<E>& r, int i, bool check) {
        float f[8];
        r.get(f);
        *reinterpret_cast<uint2*>(dst + i * GROUP * 8) = quantise8(f, inv, check);
    };
    if (full && !checked) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) put(keep[i], i, false);
    } else {
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (tid + i * GROUP < nv) put(keep[i], i, checked);
    }
#pragma unroll 1
    for (int i = KEEP; tid + i * GROUP < nv; ++i) {
        Vec8<E> r;
        r.load(src + i * STEP * rs);
        put(r, i, checked);
    }
    if (lo > b0 && s != old) {
        // the block's earlier rows move to the new scale
        const float ratio = old * inv;
        uint8_t* p = code + b0 * D;
        const int ne = (int)(lo - b0) * VR;
        for (int v = tid; v < ne; v += GROUP) {
            uint2* q = reinterpret_cast<uint2*>(p + (long long)v * 8);
            const uint2 w = *q;
            uint32_t h[4];
            e4m3x4_to_f16(w.x, h[0], h[1]);
            e4m3x4_to_f16(w.y, h[2], h[3]);
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
                f[2 * i] = t.x;
                f[2 * i + 1] = t.y;
            }
            *q = quantise8(f, ratio, false);
        }
    }
    // every lane has read the old scale: its value went through the maximum
    if (GROUP == 32)
        __syncwarp();
    if (tid == 0) *sp = s;
}

struct ReadArgs {
    const uint8_t* code[2];
    const float* scale[2];
    void* out[2];           // [B, Hkv, T, d]
    const int32_t* start;
    const int32_t* count;
    int B, Hkv, T, N, tiles;
    FastDiv R;
    int tensors;
};

// One CTA of 256 threads reads kReadRows<D> consecutive rows of one (tensor,
// sequence, head); a thread takes 8 codes at a time, all its loads first.
template <int D>
constexpr int kReadVecs = 4;
template <int D>
constexpr int kReadRows = 256 / (D / 8) * kReadVecs<D>;

template <class E, int D>
__global__ void __launch_bounds__(256) read_kernel(ReadArgs a, int* status) {
    constexpr int VR = D / 8, U = kReadVecs<D>;
    const int tile = blockIdx.x % a.tiles;
    int rest = blockIdx.x / a.tiles;
    const int j = rest % a.Hkv;
    rest /= a.Hkv;
    const int b = rest % a.B, kv = rest / a.B;
    wait_prerequisites();
    const int start = a.start[b];
    const int count = a.count ? a.count[b] : a.T;
    if (count == 0) return;
    if (start < 0 || count < 0 || count > a.T || start > a.N - count) {
        if (threadIdx.x == 0) atomicCAS(status, 0, (int)SSA_ERR_DEVICE_STATUS);
        return;
    }
    const int t0 = tile * kReadRows<D>;
    if (t0 >= count) return;
    const long long pair = (long long)b * a.Hkv + j;
    const uint8_t* code = (kv ? a.code[1] : a.code[0]) + (pair * a.N + start) * D;
    const float* sc = (kv ? a.scale[1] : a.scale[0]) + pair * (a.N / (int)a.R.d);
    E* out = static_cast<E*>(kv ? a.out[1] : a.out[0]) + pair * a.T * D;
    const int c = threadIdx.x % VR * 8, r = threadIdx.x / VR;
    uint2 w[U];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = t0 + r + u * (256 / VR);
        if (t < count) {
            w[u] = ldg64(code + (long long)t * D + c);
            s[u] = __ldg(sc + a.R.div((uint32_t)(start + t)));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = t0 + r + u * (256 / VR);
        if (t >= count) break;
        uint32_t h[4];
        e4m3x4_to_f16(w[u].x, h[0], h[1]);
        e4m3x4_to_f16(w[u].y, h[2], h[3]);
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            f[i].x *= s[u];
            f[i].y *= s[u];
        }
        E* p = out + (long long)t * D + c;
        if constexpr (sizeof(E) == 2) {
            uint4 o;
            uint32_t* ow = &o.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(f[i].x, f[i].y);
                ow[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(p) = o;
        } else {
            reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
            reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
        }
    }
}

}  // namespace ssa_q8
