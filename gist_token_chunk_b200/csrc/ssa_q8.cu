// ssa_q8.cu -- the 8-bit cache's calls: ssa_cache_append_q8, ssa_cache_read_q8,
// ssa_decode_q8, their workspace size, status word and error text.  A
// translation unit of its own (the library is compiled without relocatable
// device code), so it keeps its own status word, like the prefill.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "ssa_internal.h"
#include "ssa_q8.h"
#include "ssa_q8_cache.cuh"
#include "ssa_q8_decode.cuh"

namespace ssa_q8 {

static thread_local char g_err[256];

ssa_status fail(ssa_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}
void clear_error() { g_err[0] = 0; }

// First error since the last read; the kernels get it as an argument.
static __device__ int g_status = 0;
static __global__ void take_status_kernel(int* taken) { *taken = atomicExch(&g_status, 0); }

// Device address of g_status on the current device, looked up once per device.
static cudaError_t status_ptr(int** p) {
    static int* cached[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && __atomic_load_n(&cached[dev], __ATOMIC_ACQUIRE)) {
        *p = cached[dev];
        return cudaSuccess;
    }
    void* q = nullptr;
    e = cudaGetSymbolAddress(&q, g_status);
    if (e != cudaSuccess) return e;
    *p = static_cast<int*>(q);
    if (dev < 64) __atomic_store_n(&cached[dev], *p, __ATOMIC_RELEASE);
    return cudaSuccess;
}

// ------------------------------------------------------------ cache calls ---

// Sizes that the append and the read back share: shape's B, Hkv, d, dtype, and
// n_max as the cache's rows N.
static ssa_status check_cache(const char* who, const ssa_shape* s, int32_t R, int32_t T) {
    if (!s) return fail(SSA_ERR_INVALID_ARG, "%s: NULL shape", who);
    if (s->B < 0 || s->Hkv < 1 || s->n_max < 1 || T < 0)
        return fail(SSA_ERR_INVALID_ARG, "%s: bad sizes", who);
    if (R < 1 || s->n_max % R)
        return fail(SSA_ERR_INVALID_ARG, "%s: n_max (%d) not a multiple of R (%d)", who, s->n_max, R);
    if (s->dtype != SSA_BF16 && s->dtype != SSA_FP32)
        return fail(SSA_ERR_INVALID_ARG, "%s: unknown dtype %d", who, s->dtype);
    if (s->d != 64 && s->d != 128)
        return fail(SSA_ERR_UNSUPPORTED, "%s: d in {64, 128} only, got %d", who, s->d);
    // offsets inside a block and rows past a tile's end are 32-bit numbers
    if ((long long)R * s->d > (1 << 30) || s->n_max > INT32_MAX - 1024)
        return fail(SSA_ERR_UNSUPPORTED, "%s: R * d > 2^30, or n_max = %d too large", who, s->n_max);
    return SSA_OK;
}

template <class E, int D>
static cudaError_t launch_append(const AppendArgs& a, int* status, cudaStream_t stream) {
    const long long vectors = (long long)(a.T < a.R ? a.T : a.R) * (D / 8);
    constexpr int keep = kAppendKeep<E>;
    if (vectors <= 32 * keep)
        return launch(append_kernel<E, D, 32>, (a.items + 3) / 4, 128, 0, stream, a, status);
    if (vectors <= 64 * keep) return launch(append_kernel<E, D, 64>, a.items, 64, 0, stream, a, status);
    if (vectors <= 128 * keep)
        return launch(append_kernel<E, D, 128>, a.items, 128, 0, stream, a, status);
    return launch(append_kernel<E, D, 256>, a.items, 256, 0, stream, a, status);
}

template <class E, int D>
static cudaError_t launch_read(const ReadArgs& a, long long blocks, int* status, cudaStream_t stream) {
    return launch(read_kernel<E, D>, (unsigned)blocks, 256, 0, stream, a, status);
}

// ----------------------------------------------------------------- decode ---

struct DecodePlan {
    DecodeArgs a;
    int d, dtype;
    int attend_grid, attend_smem;
    long long score_grid;
    size_t off_keys, off_logits, off_done, off_part, bytes;
};

static ssa_status plan_decode(DecodePlan& p, const ssa_shape* s, int32_t C, int32_t g, int32_t topk) {
    if (!s) return fail(SSA_ERR_INVALID_ARG, "ssa_decode_q8: NULL shape");
    if (s->B < 1 || s->Hq < 1 || s->Hkv < 1 || s->n_max < 1)
        return fail(SSA_ERR_INVALID_ARG, "B, Hq, Hkv, n_max must be >= 1");
    if (s->Hq % s->Hkv)
        return fail(SSA_ERR_INVALID_ARG, "Hq (%d) not a multiple of Hkv (%d)", s->Hq, s->Hkv);
    if (s->Hq / s->Hkv > 16)
        return fail(SSA_ERR_UNSUPPORTED, "group size Hq/Hkv = %d > 16", s->Hq / s->Hkv);
    if (C < 1 || s->n_max % C)
        return fail(SSA_ERR_INVALID_ARG, "n_max (%d) not a multiple of C (%d)", s->n_max, C);
    if (g < 1) return fail(SSA_ERR_INVALID_ARG, "g must be >= 1");
    if (topk < 0) return fail(SSA_ERR_INVALID_ARG, "topk must be >= 0");
    if (s->dtype != SSA_BF16 && s->dtype != SSA_FP32)
        return fail(SSA_ERR_INVALID_ARG, "unknown dtype %d", s->dtype);
    if (s->d != 64 && s->d != 128)
        return fail(SSA_ERR_UNSUPPORTED, "d in {64, 128} only, got %d", s->d);
    if (g > 1024) return fail(SSA_ERR_UNSUPPORTED, "g = %d > 1024", g);
    if (topk > kMaxTopk) return fail(SSA_ERR_UNSUPPORTED, "topk = %d > %d", topk, kMaxTopk);
    const int M_max = s->n_max / C;
    // the selected chunks' bitmap in shared memory (gist rows then fit 31 bits)
    if (M_max > (1 << 19))
        return fail(SSA_ERR_UNSUPPORTED, "more than 2^19 chunks (%d) a sequence", M_max);
    if (s->n_max > INT32_MAX - 64) return fail(SSA_ERR_UNSUPPORTED, "n_max = %d too large", s->n_max);
    DecodeArgs& a = p.a;
    a = DecodeArgs{};
    a.B = s->B;
    a.Hkv = s->Hkv;
    a.Hq = s->Hq;
    a.G = s->Hq / s->Hkv;
    a.NG = (a.G + kHeads - 1) / kHeads;
    a.LG = a.G <= 4 ? 4 : 8;
    a.n_max = s->n_max;
    a.M_max = M_max;
    a.C = C;
    a.g = g;
    a.topk = topk;
    a.nch = g >= kScoreRows ? 1 : kScoreRows / g;
    if (a.nch > M_max) a.nch = M_max;
    a.tpc = (C + kTile - 1) / kTile;
    a.by_g = FastDiv((uint32_t)g);
    a.by_tpc = FastDiv((uint32_t)a.tpc);
    a.qk_scale = (float)(1.4426950408889634 / std::sqrt((double)s->d));
    p.d = s->d;
    p.dtype = s->dtype;
    const long long pairs = (long long)s->B * s->Hkv, units = pairs * a.NG;
    p.score_grid = pairs * ((M_max + a.nch - 1) / a.nch);
    // One CTA for each that is resident at a time, and up to four rounds of them
    // where each still has 64 tiles: then late CTAs even out what the rounding of
    // splits per pair leaves.  32 sequences with d = 128: 82.6 us so (two rounds), 95.5
    // with one, 91.0 from 32 tiles on; 512K batch 32.6, and 39.8 from 16 tiles on.
    const long long resident =
        (long long)ssa::sm_count() * (s->d == 64 ? kResident<64> : kResident<128>);
    const int k = topk < M_max ? topk : M_max;
    const long long tiles = ((long long)M_max * g + kTile - 1) / kTile * kGistWeight / kRawWeight +
                            (long long)k * a.tpc;
    long long rounds = units * tiles / (resident * 64);
    rounds = rounds < 1 ? 1 : rounds > 4 ? 4 : rounds;
    const long long cap = resident * rounds, grid = cap > units ? cap : units;
    // partials are one record a head and attention CTA
    if (grid > INT32_MAX || p.score_grid > INT32_MAX)
        return fail(SSA_ERR_UNSUPPORTED, "B * Hkv too large");
    p.attend_grid = (int)grid;
    const int W = s->d == 64 ? kRecord<64> : kRecord<128>;
    const int splits = grid < kMaxSplits ? (int)grid : kMaxSplits;
    const int J = s->d == 64 ? kJoin<64> : kJoin<128>;
    const int merge = kWarps * (kHeads * J > splits ? kHeads * J : splits);
    const int ring = kWarps * kStages * (int)(s->d == 64 ? sizeof(Stage<64>) : sizeof(Stage<128>));
    a.smem_sel = merge * 4 > ring ? merge * 4 : ring;
    a.smem_mask = a.smem_sel + (k + 1) * 4;
    p.attend_smem = a.smem_mask + (M_max + 31) / 32 * 4;
    a.key_stride = (M_max + 3) / 4 * 4;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    p.off_keys = 0;
    p.off_logits = up((size_t)pairs * a.key_stride * 4);
    // a last tile reads up to 15 rows past the end
    p.off_done = p.off_logits + up(((size_t)units * M_max * g + kTile) * a.LG * 4);
    p.off_part = p.off_done + up((size_t)units * 4);
    p.bytes = p.off_part + up((size_t)grid * kHeads * W * 4);
    return SSA_OK;
}

// Function attributes, once per device: the attention's shared memory (at most
// 120 KB: ring, selection, bitmap), and one split of the SM's memory for it and
// the selection, so that its CTAs may join the selection's.  The scores keep the
// default: next to attention CTAs that already copy gists they ran longer.
template <class E, int D>
static cudaError_t prepare_kernels() {
    static int done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && __atomic_load_n(&done[dev], __ATOMIC_ACQUIRE))) return e;
    const void* all[] = {(const void*)select_kernel, (const void*)attend_kernel<E, D>};
    for (const void* f : all) {
        e = cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
    }
    e = cudaFuncSetAttribute(attend_kernel<E, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             160 * 1024);
    if (e == cudaSuccess && dev < 64) __atomic_store_n(&done[dev], 1, __ATOMIC_RELEASE);
    return e;
}

template <class E, int D>
static cudaError_t launch_decode(const DecodePlan& p, int* status, cudaStream_t stream) {
    const DecodeArgs& a = p.a;
    cudaError_t e = prepare_kernels<E, D>();
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)p.score_grid;
    const size_t best = (size_t)a.nch * 8;
    e = launch(a.NG == 1 ? score_kernel<E, D, 1> : score_kernel<E, D, 2>, grid, 128, best, stream, a);
    if (e != cudaSuccess) return e;
    if (a.topk > 0) {
        // One warp needs no barrier, and more take at least four: CTAs of two warps
        // started and ran late next to the attention's (128K batch: 29.2 us a step
        // with two, 26.3 with four; 32K batch 24.2 with one, 24.8 with four).
        int warps = (a.M_max + 32 * kSelectKeys - 1) / (32 * kSelectKeys);
        warps = warps == 1 ? 1 : warps < 4 ? 4 : warps;
        const bool wide = 32 * warps > kSelThreads;
        e = launch(select_kernel, (unsigned)(a.B * a.Hkv), wide ? kSelThreads : 32 * warps,
                   wide ? 2048 * 4 : 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    return launch(attend_kernel<E, D>, (unsigned)p.attend_grid, 32 * kWarps, p.attend_smem, stream, a,
                  status);
}

}  // namespace ssa_q8

using namespace ssa_q8;

extern "C" {

SSA_API ssa_status ssa_cache_append_q8(const ssa_shape* shape, int32_t T, int32_t R,
                                       const void* k_new, const int64_t* k_strides,
                                       const void* v_new, const int64_t* v_strides,
                                       const int32_t* start, const int32_t* count, uint8_t* k_q8,
                                       uint8_t* v_q8, float* k_scale, float* v_scale,
                                       cudaStream_t stream) {
    clear_error();
    ssa_status st = check_cache("ssa_cache_append_q8", shape, R, T);
    if (st != SSA_OK) return st;
    const ssa_shape& s = *shape;
    if (s.B == 0 || T == 0) return SSA_OK;
    if (!k_new || !k_strides || !start || !k_q8 || !k_scale ||
        (v_new && (!v_strides || !v_q8 || !v_scale)))
        return fail(SSA_ERR_INVALID_ARG, "ssa_cache_append_q8: NULL pointer");
    AppendArgs a = {};
    a.tensors = v_new ? 2 : 1;
    const int e = s.dtype == SSA_BF16 ? 2 : 4;
    const void* x[2] = {k_new, v_new};
    const int64_t* xs[2] = {k_strides, v_strides};
    uint8_t* code[2] = {k_q8, v_q8};
    float* scale[2] = {k_scale, v_scale};
    for (int i = 0; i < a.tensors; ++i) {
        if (!aligned(x[i], 16) || !aligned(code[i], 16) || !aligned(scale[i], 4))
            return fail(SSA_ERR_INVALID_ARG, "ssa_cache_append_q8: misaligned pointer");
        for (int n = 0; n < 3; ++n) {
            if ((xs[i][n] * e) % 16)
                return fail(SSA_ERR_UNSUPPORTED,
                            "ssa_cache_append_q8: strides must be multiples of 16 bytes");
            a.xs[i][n] = xs[i][n];
        }
        a.x[i] = x[i];
        a.code[i] = code[i];
        a.scale[i] = scale[i];
    }
    if (!aligned(start, 4) || !aligned(count, 4))
        return fail(SSA_ERR_INVALID_ARG, "ssa_cache_append_q8: misaligned pointer");
    a.start = start;
    a.count = count;
    a.B = s.B;
    a.Hkv = s.Hkv;
    a.T = T;
    a.R = R;
    a.N = s.n_max;
    const long long most = ((long long)T + R - 2) / R + 1, have = s.n_max / R;
    a.nblk = (int)(most < have ? most : have);
    const long long items = (long long)a.tensors * s.B * s.Hkv * a.nblk;
    if (items > INT32_MAX - 4) return fail(SSA_ERR_UNSUPPORTED, "ssa_cache_append_q8: too many blocks");
    a.items = (uint32_t)items;
    a.by_heads = FastDiv((uint32_t)s.Hkv);
    a.by_blocks = FastDiv((uint32_t)a.nblk);
    a.by_rows = FastDiv((uint32_t)R);
    int* status = nullptr;
    cudaError_t err = status_ptr(&status);
    if (err == cudaSuccess) {
        if (s.dtype == SSA_BF16)
            err = s.d == 64 ? launch_append<__nv_bfloat16, 64>(a, status, stream)
                            : launch_append<__nv_bfloat16, 128>(a, status, stream);
        else
            err = s.d == 64 ? launch_append<float, 64>(a, status, stream)
                            : launch_append<float, 128>(a, status, stream);
    }
    if (err != cudaSuccess)
        return fail(SSA_ERR_CUDA, "ssa_cache_append_q8: %s", cudaGetErrorString(err));
    return SSA_OK;
}

SSA_API ssa_status ssa_cache_read_q8(const ssa_shape* shape, int32_t T, int32_t R,
                                     const uint8_t* k_q8, const uint8_t* v_q8,
                                     const float* k_scale, const float* v_scale,
                                     const int32_t* start, const int32_t* count, void* k_out,
                                     void* v_out, cudaStream_t stream) {
    clear_error();
    ssa_status st = check_cache("ssa_cache_read_q8", shape, R, T);
    if (st != SSA_OK) return st;
    const ssa_shape& s = *shape;
    if (s.B == 0 || T == 0) return SSA_OK;
    if (!k_q8 || !k_scale || !start || !k_out || (v_q8 && (!v_scale || !v_out)))
        return fail(SSA_ERR_INVALID_ARG, "ssa_cache_read_q8: NULL pointer");
    const void* wide[] = {k_q8, v_q8, k_out, v_out};
    const void* word[] = {k_scale, v_scale, start, count};
    for (const void* q : wide)
        if (!aligned(q, 16)) return fail(SSA_ERR_INVALID_ARG, "ssa_cache_read_q8: misaligned pointer");
    for (const void* q : word)
        if (!aligned(q, 4)) return fail(SSA_ERR_INVALID_ARG, "ssa_cache_read_q8: misaligned pointer");
    ReadArgs a = {};
    a.code[0] = k_q8;
    a.code[1] = v_q8;
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    a.out[0] = k_out;
    a.out[1] = v_out;
    a.start = start;
    a.count = count;
    a.B = s.B;
    a.Hkv = s.Hkv;
    a.T = T;
    a.N = s.n_max;
    a.R = FastDiv((uint32_t)R);
    a.tensors = v_q8 ? 2 : 1;
    const int rows = s.d == 64 ? kReadRows<64> : kReadRows<128>;
    a.tiles = (T - 1) / rows + 1;
    const long long blocks = (long long)a.tiles * a.tensors * s.B * s.Hkv;
    if (blocks > INT32_MAX) return fail(SSA_ERR_UNSUPPORTED, "ssa_cache_read_q8: too many rows");
    int* status = nullptr;
    cudaError_t err = status_ptr(&status);
    if (err == cudaSuccess) {
        if (s.dtype == SSA_BF16)
            err = s.d == 64 ? launch_read<__nv_bfloat16, 64>(a, blocks, status, stream)
                            : launch_read<__nv_bfloat16, 128>(a, blocks, status, stream);
        else
            err = s.d == 64 ? launch_read<float, 64>(a, blocks, status, stream)
                            : launch_read<float, 128>(a, blocks, status, stream);
    }
    if (err != cudaSuccess)
        return fail(SSA_ERR_CUDA, "ssa_cache_read_q8: %s", cudaGetErrorString(err));
    return SSA_OK;
}

SSA_API ssa_status ssa_workspace_size_q8(const ssa_shape* shape, int32_t C, int32_t g, int32_t topk,
                                         size_t* bytes) {
    clear_error();
    if (!bytes) return fail(SSA_ERR_INVALID_ARG, "bytes is NULL");
    DecodePlan p;
    ssa_status st = plan_decode(p, shape, C, g, topk);
    if (st != SSA_OK) return st;
    *bytes = p.bytes;
    return SSA_OK;
}

SSA_API ssa_status ssa_decode_q8(const ssa_shape* shape, const void* q, const uint8_t* k_raw,
                                 const uint8_t* v_raw, const uint8_t* k_gist,
                                 const uint8_t* v_gist, const float* k_raw_scale,
                                 const float* v_raw_scale, const float* k_gist_scale,
                                 const float* v_gist_scale, const int32_t* seq_lens, int32_t C,
                                 int32_t g, int32_t topk, float* out, int32_t* sel_idx, void* ws,
                                 size_t ws_bytes, cudaStream_t stream) {
    clear_error();
    DecodePlan p;
    ssa_status st = plan_decode(p, shape, C, g, topk);
    if (st != SSA_OK) return st;
    const void* wide[] = {q, k_raw, v_raw, k_gist, v_gist};
    const void* word[] = {k_raw_scale, v_raw_scale, k_gist_scale, v_gist_scale, seq_lens, out};
    for (const void* x : wide) {
        if (!x) return fail(SSA_ERR_INVALID_ARG, "a required pointer is NULL");
        if (!aligned(x, 16)) return fail(SSA_ERR_UNSUPPORTED, "tensors must be 16-byte aligned");
    }
    for (const void* x : word) {
        if (!x) return fail(SSA_ERR_INVALID_ARG, "a required pointer is NULL");
        if (!aligned(x, 4)) return fail(SSA_ERR_INVALID_ARG, "misaligned pointer");
    }
    if (topk > 0 && (!sel_idx || !aligned(sel_idx, 4)))
        return fail(SSA_ERR_INVALID_ARG, "sel_idx is NULL or misaligned");
    void* own = nullptr;
    cudaError_t e;
    if (ws == nullptr) {
        if (ws_bytes != 0) return fail(SSA_ERR_WORKSPACE, "ws is NULL but ws_bytes != 0");
    } else if (ws_bytes < p.bytes) {
        return fail(SSA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, p.bytes);
    } else if (!aligned(ws, 256)) {
        return fail(SSA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    }
    int* status = nullptr;
    e = status_ptr(&status);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "ssa_decode_q8: %s", cudaGetErrorString(e));
    if (ws == nullptr) {
        e = cudaMallocAsync(&own, p.bytes, stream);
        if (e != cudaSuccess)
            return fail(SSA_ERR_CUDA, "cudaMallocAsync(workspace): %s", cudaGetErrorString(e));
        ws = own;
    }
    DecodeArgs& a = p.a;
    char* base = static_cast<char*>(ws);
    a.keys = reinterpret_cast<uint32_t*>(base + p.off_keys);
    a.logits = reinterpret_cast<float*>(base + p.off_logits);
    a.done = reinterpret_cast<int*>(base + p.off_done);
    a.part = reinterpret_cast<float*>(base + p.off_part);
    a.q = q;
    a.k_raw = k_raw;
    a.v_raw = v_raw;
    a.k_gist = k_gist;
    a.v_gist = v_gist;
    a.k_raw_s = k_raw_scale;
    a.v_raw_s = v_raw_scale;
    a.k_gist_s = k_gist_scale;
    a.v_gist_s = v_gist_scale;
    a.seq_lens = seq_lens;
    a.out = out;
    a.sel = sel_idx;
    if (p.dtype == SSA_BF16)
        e = p.d == 64 ? launch_decode<__nv_bfloat16, 64>(p, status, stream)
                      : launch_decode<__nv_bfloat16, 128>(p, status, stream);
    else
        e = p.d == 64 ? launch_decode<float, 64>(p, status, stream)
                      : launch_decode<float, 128>(p, status, stream);
    if (own) cudaFreeAsync(own, stream);
    if (e != cudaSuccess) return fail(SSA_ERR_CUDA, "ssa_decode_q8: %s", cudaGetErrorString(e));
    return SSA_OK;
}

SSA_API ssa_status ssa_cache_get_status(int32_t* host_code, cudaStream_t stream) {
    clear_error();
    if (!host_code) return fail(SSA_ERR_INVALID_ARG, "ssa_cache_get_status: NULL output");
    // a word of the call's own: readers on several streams never see each other's
    int v = 0, *taken = nullptr;
    cudaError_t e = cudaMallocAsync(reinterpret_cast<void**>(&taken), sizeof(int), stream);
    if (e == cudaSuccess) {
        take_status_kernel<<<1, 1, 0, stream>>>(taken);
        e = cudaGetLastError();
        if (e == cudaSuccess)
            e = cudaMemcpyAsync(&v, taken, sizeof(int), cudaMemcpyDeviceToHost, stream);
        cudaFreeAsync(taken, stream);
    }
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess)
        return fail(SSA_ERR_CUDA, "ssa_cache_get_status: %s", cudaGetErrorString(e));
    *host_code = v;
    return SSA_OK;
}

SSA_API const char* ssa_cache_last_error(void) { return g_err; }

}  // extern "C"
