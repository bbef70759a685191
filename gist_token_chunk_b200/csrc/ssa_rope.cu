// ssa_rope.cu -- rotary positions: ssa_rope_freqs (host) and ssa_rope.
//
// Pair i of a row at position p turns by the angle w = p f_i:
//     y_a = s (x_a cos w - x_b sin w),   y_b = s (x_b cos w + x_a sin w)
// with (a, b) = (i, i + r/2) in the half layout and (2i, 2i + 1) in the
// interleaved one, r the rotated dims; the other d - r dims are copied.
//
// Bound by HBM: every element is read and written once, 3 flop an element.
// 16K tokens of 40 heads of 128 take 60.9 us, 0.84 of the copy's rate; a decode step's
// rows (8 sequences) 2.3 us.
// A thread keeps one (sequence, row, place in the row) and walks the heads, so
// its angles' cosines and sines are computed once, stay in registers and serve
// every head; with few rows the heads are split over more threads instead.
// The angle is reduced to the fraction of a turn in twice 64 bits: at positions near 2^31 a
// product in 64 leaves 22 bits of the fraction, one in 32 none.  The rest is fp32 (the
// fraction's rounding to it moves cosine and sine by 1.6 * 2^-24 at most; correcting them by
// what it left took 61.7 us in place of 61.3 on the prompt below), rounded once on the way out.
#include <cmath>

#include "ssa_internal.h"
#include "ssa_q8.h"

namespace ssa_rope_k {

using ssa_q8::fail;
using ssa_q8::wait_prerequisites;

struct Tensor {
    const void* in;
    void* out;
    long long is[3], os[3];  // strides in elements: sequence, head, row
};

struct Args {
    Tensor t[2];  // queries, keys
    int Hq, H;    // query heads, all heads
    int B, T, d, rd, items, rot_items;
    long long n;             // B * T * items
    int heads_per_thread;
    const int32_t* pos;
    int pos_rows;            // 1: pos[b, t]; 0: pos[b] + t
    const double* freqs;
    float scale, sign;
};

template <class E, int V>
struct alignas(sizeof(E) * V) Pack {
    E e[V];
};

// Cosine and sine of the angle p f, |p| < 2^33: f / 2 pi is g + gl, 106 bits, and p g + (its
// rounding error) + p gl less whole turns is the fraction of a turn, to 2^-53 of one.
__device__ __forceinline__ void turn(double p, double f, float& c, float& s) {
    constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;  // 1 / 2 pi
    const double g = f * kInv, gl = fma(f, kInv, -g) + f * kInvLow;
    const double t = p * g;
    const double fraction = (t - rint(t)) + fma(p, gl, fma(p, g, -t));
    sincospif((float)(2.0 * fraction), &s, &c);
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// One item is V pairs: in the half layout a run of V dims of each half, in the
// interleaved one a run of 2 V dims; the copied dims, d - r, are taken the same way.
// So neighbouring lanes' 16 bytes are neighbours in memory in either layout (two
// runs side by side would leave each access half of every 32-byte sector).
// kScattered is the interleaved layout by single elements, for rows that do not
// start on a pair's boundary.
enum Mode { kHalf, kPairs, kScattered };
template <class E, int V, int MODE>
__global__ void __launch_bounds__(256) rope_kernel(Args a) {
    constexpr int RUN = MODE == kPairs ? 2 * V : V, RUNS = MODE == kPairs ? 1 : 2;
    static_assert(MODE != kScattered || V == 1, "single elements");
    using P = Pack<E, RUN>;
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    if (idx >= a.n) return;
    const int item = (int)(idx % a.items);
    const long long bt = idx / a.items;
    const int t = (int)(bt % a.T), b = (int)(bt / a.T);
    const bool rot = item < a.rot_items;
    const int i0 = rot ? item : item - a.rot_items;
    const int o0 = (rot ? 0 : a.rd) + i0 * (MODE == kScattered ? 2 : RUN);
    const int o1 = MODE == kScattered ? o0 + 1 : o0 + (rot ? a.rd / 2 : (a.d - a.rd + 1) / 2);
    const bool second = RUNS == 2 && o1 < a.d;  // of an odd number of copied dims, not the last

    constexpr int U = 4;  // heads in flight
    P x[U][RUNS];
    const int h0 = blockIdx.y * a.heads_per_thread;
    const int h1 = min(a.H, h0 + a.heads_per_thread);
    auto base = [&](int i, bool out) {
        const Tensor& q = a.t[i];
        const long long* s = out ? q.os : q.is;
        return static_cast<E*>(out ? q.out : const_cast<void*>(q.in)) + b * s[0] + t * s[2];
    };
    auto load = [&](const E* p, P (&r)[RUNS]) {
        r[0] = *reinterpret_cast<const P*>(p + o0);
        if (second) r[RUNS - 1] = *reinterpret_cast<const P*>(p + o1);
    };
    wait_prerequisites();
    // the first heads' loads go out before the angles are computed
    const int part0 = h0 < a.Hq ? 0 : 1;
    {
        const int skip = part0 ? a.Hq : 0, end = part0 ? a.H : min(a.Hq, h1);
        const long long step = a.t[part0].is[1];
        const E* p = base(part0, false) + (h0 - skip) * step;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h0 + u < min(end, h1)) load(p + u * step, x[u]);
    }
    float c[V], s[V];
    if (rot) {
        const double p = a.pos_rows ? (double)a.pos[(long long)b * a.T + t]
                                    : (double)a.pos[b] + (double)t;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float sn, cs;
            turn(p, a.freqs[i0 * V + i], cs, sn);
            c[i] = a.scale * cs;
            s[i] = a.scale * (a.sign * sn);
        }
    }
#pragma unroll 1
    for (int part = part0; part < 2; ++part) {
        // this thread's heads of the queries, then of the keys
        const int skip = part ? a.Hq : 0;
        const int lo = max(h0, skip), hi = min(h1, part ? a.H : a.Hq);
        if (lo >= hi) continue;
        const long long si = a.t[part].is[1], so = a.t[part].os[1];
        const E* in = base(part, false) + (lo - skip) * si;
        E* out = base(part, true) + (lo - skip) * so;
#pragma unroll 1
        for (int h = lo; h < hi; h += U, in += U * si, out += U * so) {
            if (h != h0) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h + u < hi) load(in + u * si, x[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h + u >= hi) break;
                if (rot) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        E& ea = x[u][0].e[RUNS == 2 ? i : 2 * i];
                        E& eb = RUNS == 2 ? x[u][RUNS - 1].e[i] : x[u][0].e[(2 * i + 1) % RUN];
                        const float p = to_f(ea), q = to_f(eb);
                        from_f(ea, p * c[i] - q * s[i]);
                        from_f(eb, q * c[i] + p * s[i]);
                    }
                }
                E* p = out + u * so;
                *reinterpret_cast<P*>(p + o0) = x[u][0];
                if (second) *reinterpret_cast<P*>(p + o1) = x[u][RUNS - 1];
            }
        }
    }
}

template <class E, int V>
cudaError_t launch_v(const Args& a, int mode, dim3 grid, cudaStream_t stream) {
    if (mode == kHalf) return ssa_q8::launch(rope_kernel<E, V, kHalf>, grid, 256, 0, stream, a);
    if constexpr (2 * V * sizeof(E) <= 16)
        if (mode == kPairs) return ssa_q8::launch(rope_kernel<E, V, kPairs>, grid, 256, 0, stream, a);
    return ssa_q8::launch(rope_kernel<E, 1, kScattered>, grid, 256, 0, stream, a);
}

// Whether items of v pairs fit the layout, the strides and the addresses.
bool fits(const Args& a, int e, int v, bool half, bool copies) {
    const int run = half ? v : 2 * v;
    if ((a.rd / 2) % v) return false;
    if (copies && ((a.d - a.rd) % (2 * v) || a.rd % run)) return false;
    const long long bytes = (long long)e * run;
    for (int i = 0; i < 2; ++i) {
        if (i == 1 && a.H == a.Hq) break;
        const Tensor& t = a.t[i];
        if (!ssa_q8::aligned(t.in, (unsigned)bytes) || !ssa_q8::aligned(t.out, (unsigned)bytes))
            return false;
        for (int k = 0; k < 3; ++k)
            if ((t.is[k] * e) % bytes || (t.os[k] * e) % bytes) return false;
    }
    return true;
}

}  // namespace ssa_rope_k

using namespace ssa_rope_k;

extern "C" {

SSA_API ssa_status ssa_rope_freqs(int32_t rotary_dim, double base, int32_t scaling, double factor,
                                  double low, double high, double original_length,
                                  double* freqs_host, float* scale) {
    ssa_q8::clear_error();
    if (!freqs_host || !scale) return fail(SSA_ERR_INVALID_ARG, "ssa_rope_freqs: NULL output");
    if (rotary_dim < 2 || rotary_dim % 2 || !(base > 1.0) || !std::isfinite(base))
        return fail(SSA_ERR_INVALID_ARG, "ssa_rope_freqs: need an even rotary_dim >= 2, base > 1");
    if (scaling < SSA_ROPE_PLAIN || scaling > SSA_ROPE_RAMPED)
        return fail(SSA_ERR_INVALID_ARG, "ssa_rope_freqs: scaling = %d is not a scaling", scaling);
    if (scaling != SSA_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor)))
        return fail(SSA_ERR_INVALID_ARG, "ssa_rope_freqs: need a finite factor >= 1");
    if (scaling >= SSA_ROPE_BANDED &&
        !(low > 0.0 && high > low && std::isfinite(high) && original_length >= 1.0 &&
          std::isfinite(original_length)))
        return fail(SSA_ERR_INVALID_ARG,
                    "ssa_rope_freqs: need 0 < low < high and original_length >= 1");
    const double two_pi = 6.283185307179586476925;
    const int half = rotary_dim / 2;
    // RAMPED: the pair that makes `turns` turns over the original length
    auto pair_of = [&](double turns) {
        return rotary_dim * std::log(original_length / (turns * two_pi)) / (2.0 * std::log(base));
    };
    double first = 0.0, last = 0.0;
    if (scaling == SSA_ROPE_RAMPED) {
        first = std::floor(pair_of(high));
        last = std::ceil(pair_of(low));
        if (first < 0.0) first = 0.0;
        // past the last pair, r/2 - 1, where that makes more than `low` turns itself
        if (last > rotary_dim - 1) last = rotary_dim - 1;
        if (last <= first) last = first + 0.001;
    }
    for (int i = 0; i < half; ++i) {
        double f = std::pow(base, -2.0 * i / rotary_dim);
        if (scaling == SSA_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == SSA_ROPE_BANDED) {
            const double turns = original_length * f / two_pi;
            double keep = (turns - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = keep * f + (1.0 - keep) * f / factor;
        } else if (scaling == SSA_ROPE_RAMPED) {
            double slow = (i - first) / (last - first);
            slow = slow < 0.0 ? 0.0 : slow > 1.0 ? 1.0 : slow;
            f = (1.0 - slow) * f + slow * f / factor;
        }
        freqs_host[i] = f;
    }
    *scale = scaling == SSA_ROPE_RAMPED ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return SSA_OK;
}

SSA_API ssa_status ssa_rope(const ssa_shape* shape, int32_t T, const void* q,
                            const int64_t* q_strides, void* q_out, const int64_t* q_out_strides,
                            const void* k, const int64_t* k_strides, void* k_out,
                            const int64_t* k_out_strides, const int32_t* pos, int32_t pos_rows,
                            const double* freqs, int32_t rotary_dim, int32_t layout, float scale,
                            int32_t inverse, cudaStream_t stream) {
    ssa_q8::clear_error();
    if (!shape) return fail(SSA_ERR_INVALID_ARG, "ssa_rope: NULL shape");
    const ssa_shape& s = *shape;
    if (s.B < 0 || s.Hq < 1 || T < 0 || s.d < 2 || (k && s.Hkv < 1))
        return fail(SSA_ERR_INVALID_ARG, "ssa_rope: bad sizes");
    if (s.dtype != SSA_BF16 && s.dtype != SSA_FP32)
        return fail(SSA_ERR_INVALID_ARG, "ssa_rope: unknown dtype %d", s.dtype);
    if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > s.d)
        return fail(SSA_ERR_INVALID_ARG, "ssa_rope: rotary_dim = %d is not even in [2, %d]",
                    rotary_dim, s.d);
    if (layout != SSA_ROPE_HALF && layout != SSA_ROPE_INTERLEAVED)
        return fail(SSA_ERR_INVALID_ARG, "ssa_rope: layout = %d is not a layout", layout);
    if ((long long)s.Hq + (k ? s.Hkv : 0) > INT32_MAX - 1024)
        return fail(SSA_ERR_UNSUPPORTED, "ssa_rope: more than 2^31 - 1025 heads");
    if (s.B == 0 || T == 0) return SSA_OK;
    if (!q || !q_out || !q_strides || !q_out_strides || !pos || !freqs ||
        (k && (!k_out || !k_strides || !k_out_strides)))
        return fail(SSA_ERR_INVALID_ARG, "ssa_rope: NULL pointer");
    const int e = s.dtype == SSA_BF16 ? 2 : 4;
    if (!ssa_q8::aligned(pos, 4) || !ssa_q8::aligned(freqs, 8) || !ssa_q8::aligned(q, e) ||
        !ssa_q8::aligned(q_out, e) || (k && (!ssa_q8::aligned(k, e) || !ssa_q8::aligned(k_out, e))))
        return fail(SSA_ERR_INVALID_ARG, "ssa_rope: misaligned pointer");

    Args a = {};
    a.t[0] = {q, q_out, {q_strides[0], q_strides[1], q_strides[2]},
              {q_out_strides[0], q_out_strides[1], q_out_strides[2]}};
    if (k)
        a.t[1] = {k, k_out, {k_strides[0], k_strides[1], k_strides[2]},
                  {k_out_strides[0], k_out_strides[1], k_out_strides[2]}};
    // in place: the dims that do not turn are where they belong
    bool copies = false;
    for (int i = 0; i < (k ? 2 : 1); ++i) {
        bool same = a.t[i].in == a.t[i].out;
        for (int n = 0; n < 3; ++n) same = same && a.t[i].is[n] == a.t[i].os[n];
        copies = copies || !same;
    }
    copies = copies && rotary_dim < s.d;
    a.Hq = s.Hq;
    a.H = s.Hq + (k ? s.Hkv : 0);
    a.B = s.B;
    a.T = T;
    a.d = s.d;
    a.rd = rotary_dim;
    a.pos = pos;
    a.pos_rows = pos_rows ? 1 : 0;
    a.freqs = freqs;
    a.scale = scale;
    a.sign = inverse ? -1.0f : 1.0f;
    const bool half = layout == SSA_ROPE_HALF;
    int v = (half ? 16 : 8) / e;  // widest run: 16 bytes
    while (v > 1 && !fits(a, e, v, half, copies)) v /= 2;
    const int mode = half ? kHalf : fits(a, e, v, half, copies) ? kPairs : kScattered;
    a.rot_items = rotary_dim / 2 / v;
    a.items = a.rot_items + (copies ? (s.d - rotary_dim + 2 * v - 1) / (2 * v) : 0);
    a.n = (long long)s.B * T * a.items;
    const long long blocks = (a.n + 255) / 256;
    if (blocks > INT32_MAX) return fail(SSA_ERR_UNSUPPORTED, "ssa_rope: too many rows");
    // heads split over threads until there are eight CTAs an SM; fewer are resident: two
    // (bf16 half layout, 117 registers a thread), four (runs of 16 bytes otherwise) to six
    const long long want = (long long)ssa::sm_count() * 8;
    long long split = blocks >= want ? 1 : (want + blocks - 1) / blocks;
    if (split > a.H) split = a.H;
    if (split > 65535) split = 65535;
    a.heads_per_thread = (int)((a.H + split - 1) / split);
    const dim3 grid((unsigned)blocks, (unsigned)((a.H + a.heads_per_thread - 1) / a.heads_per_thread));
    cudaError_t err;
    if (s.dtype == SSA_BF16)
        err = v == 8   ? launch_v<__nv_bfloat16, 8>(a, mode, grid, stream)
              : v == 4 ? launch_v<__nv_bfloat16, 4>(a, mode, grid, stream)
              : v == 2 ? launch_v<__nv_bfloat16, 2>(a, mode, grid, stream)
                       : launch_v<__nv_bfloat16, 1>(a, mode, grid, stream);
    else
        err = v == 4   ? launch_v<float, 4>(a, mode, grid, stream)
              : v == 2 ? launch_v<float, 2>(a, mode, grid, stream)
                       : launch_v<float, 1>(a, mode, grid, stream);
    if (err != cudaSuccess) return fail(SSA_ERR_CUDA, "ssa_rope: %s", cudaGetErrorString(err));
    return SSA_OK;
}

}  // extern "C"
