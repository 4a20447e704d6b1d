// zc_optim.hip -- the gradient norm and the AdamW step over many tensors
// (zc_grad_norm, zc_adamw; the definitions are in zc_ops.h).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "zc_ops.h"
#include "zc_device.h"

namespace {

using namespace zcd;

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kLanes;
constexpr uint32_t kMaxBlocks = (1u << 24) - 1;    // workgroups of a launch (2^32 threads)

// PER neighbouring values (4 or 8) at p[i ..], zeros past n.
template <bool STREAM, int PER, class T>
__device__ inline void load_run(const T* p, int64_t i, int64_t n, float (&f)[PER])
{
    constexpr int N = Word<T>::N;
    if (i + PER <= n) {
        if constexpr (PER < N) {
            float w[N];
            const u32x2 h = load8<STREAM>(p + i);
            Word<T>::unpack(u32x4{h[0], h[1], 0, 0}, w);
#pragma unroll
            for (int c = 0; c < PER; ++c)
                f[c] = w[c];
        } else {
#pragma unroll
            for (int h = 0; h < PER / N; ++h) {
                float w[N];
                Word<T>::unpack(load16<STREAM>(p + i + h * N), w);
#pragma unroll
                for (int c = 0; c < N; ++c)
                    f[h * N + c] = w[c];
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < PER; ++c)
            f[c] = 0.0f;
        if (i < n) {                               // the one lane that holds the end
#pragma unroll
            for (int c = 0; c < PER; ++c)
                if (i + c < n)
                    f[c] = widen(p[i + c]);
        }
    }
}

template <bool STREAM, int PER, class T>
__device__ inline void store_run(T* p, int64_t i, int64_t n, const float (&f)[PER])
{
    constexpr int N = Word<T>::N;
    if (i + PER <= n) {
        if constexpr (PER < N) {
            float w[N] = {};
#pragma unroll
            for (int c = 0; c < PER; ++c)
                w[c] = f[c];
            const u32x4 h = Word<T>::pack(w);
            store8<STREAM>(p + i, u32x2{h[0], h[1]});
        } else {
#pragma unroll
            for (int h = 0; h < PER / N; ++h) {
                float w[N];
#pragma unroll
                for (int c = 0; c < N; ++c)
                    w[c] = f[h * N + c];
                store16<STREAM>(p + i + h * N, Word<T>::pack(w));
            }
        }
    } else if (i < n) {
#pragma unroll
        for (int c = 0; c < PER; ++c)
            if (i + c < n)
                p[i + c] = static_cast<T>(f[c]);
    }
}

// Index of the tensor that holds workgroup b: the last whose first workgroup
// is at most b, one entry per lane and ballot.
template <int M>
__device__ inline int tensor_of(const uint32_t (&first)[M], uint32_t b)
{
    int at = -1;
#pragma unroll
    for (int i = 0; i < M; i += kLanes) {
        const int c = i + (threadIdx.x & (kLanes - 1));
        at += __popcll(__ballot((c < M ? first[c] : ~0u) <= b));
    }
    return __builtin_amdgcn_readfirstlane(at);
}

// ------------------------------------------------------------ gradient norm

// A launch's arguments hold its table: up to 4 KB with the 256 hidden bytes,
// or a short one where that will do (a launch costs the host 1.1 us more with
// 3.3 KB of arguments than with few).
constexpr int kNormTensors = 238;
constexpr int kNormShort = 32;
constexpr int kNormWords = 8;                      // 16-byte words per thread, all in flight at once
constexpr int kNormChunkBytes = kBlock * kNormWords * 16;
constexpr int kFinishBlock = 1024;
constexpr int kFinishWaves = kFinishBlock / kLanes;
constexpr int kPieceBytes = kLanes * kNormWords * 16;
constexpr int64_t kNormOne = 2 * kFinishWaves;     // pieces that one workgroup sums alone

template <int M>
struct NormTable {
    const void* data[M];
    uint32_t first[M];                             // ~0 past the last tensor
    uint32_t last_n[M];                            // values of the tensor's last chunk
};

static_assert(sizeof(NormTable<kNormTensors>) + 16 + 256 <= 4096, "kernel arguments");

// One piece (BYTES of one tensor, the last may be shorter) of a launch's list.
template <class T, int BYTES>
struct Chunk {
    const T* p;
    int64_t n;
    template <int M>
    __device__ Chunk(const NormTable<M>& tab, uint32_t b, uint32_t blocks)
    {
        constexpr int64_t kValues = BYTES / sizeof(T);
        const int i = tensor_of(tab.first, b);
        const uint32_t first = tab.first[i];
        const uint32_t next = i + 1 < M ? tab.first[i + 1] : ~0u;
        n = b + 1 == (next < blocks ? next : blocks) ? tab.last_n[i] : kValues;
        p = static_cast<const T*>(tab.data[i]) + static_cast<int64_t>(b - first) * kValues;
    }
};

// WORDS 16-byte words of a piece, `step` words apart from word `at` on.  The
// word that holds the end begins early, in its neighbour's, and a lane past
// the end takes the piece's first, so that no load waits for a branch.  (A
// piece shorter than a word is read value by value, into the first word of
// its lane 0.)
template <bool STREAM, int WORDS, class T, int BYTES>
__device__ inline void load_words(const Chunk<T, BYTES>& c, int at, int step, u32x4 (&w)[WORDS])
{
    constexpr int N = Word<T>::N;
    if (c.n >= N) {
#pragma unroll
        for (int s = 0; s < WORDS; ++s) {
            const int64_t i = static_cast<int64_t>(at + s * step) * N;
            w[s] = load16<STREAM>(c.p + (i + N <= c.n ? i : i < c.n ? c.n - N : 0));
        }
    } else {
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] = i < c.n ? widen(c.p[i]) : 0.0f;
        w[0] = Word<T>::pack(f);
    }
}

// Sum of their squares in fp64: no gradient's square overflows, and the
// order of additions hardly ever shows in the fp32 result.
template <int WORDS, class T, int BYTES>
__device__ inline double squares(const Chunk<T, BYTES>& c, int at, int step, const u32x4 (&w)[WORDS])
{
    constexpr int N = Word<T>::N;
    double sum = 0.0;
#pragma unroll
    for (int s = 0; s < WORDS; ++s) {
        const int64_t i = static_cast<int64_t>(at + s * step) * N;
        if (i >= c.n)
            continue;
        float f[N];
        Word<T>::unpack(w[s], f);
        if (i + N > c.n && c.n >= N) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                f[k] = c.n - N + k < i ? 0.0f : f[k];
        }
#pragma unroll
        for (int k = 0; k < N; ++k)
            sum = fma(static_cast<double>(f[k]), static_cast<double>(f[k]), sum);
    }
    return sum;
}

// Sum over the workgroup's waves, for thread 0.
template <int WAVES>
__device__ inline double block_sum(double sum)
{
    __shared__ double s_part[WAVES];
    sum = reduce_sum<kLanes>(sum);
    if ((threadIdx.x & (kLanes - 1)) == 0)
        s_part[threadIdx.x / kLanes] = sum;
    __syncthreads();
    double all = s_part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
        all += s_part[w];
    return all;
}

__device__ inline void write_norm(double all, float max_norm, float* out)
{
    const float norm = static_cast<float>(sqrt(all));
    float clip = 1.0f;
    if (max_norm > 0.0f)
        clip = fminf(1.0f, max_norm / (norm + 1e-6f));
    if (!(norm <= 3.402823466e38f))
        clip = __builtin_nanf("");
    out[0] = norm;
    out[1] = clip;
}

// Bound by memory: 239 MB of bf16 in 200 tensors in 38 us (6.2 TB/s), 268 MB
// of fp32 in 41 us (6.5); a read of one large buffer reaches 6.8 to 7.0.
template <class T, bool STREAM, int M>
__global__ __launch_bounds__(kBlock) void zc_norm_kernel(NormTable<M> tab, uint32_t blocks, double* __restrict__ partial)
{
    const Chunk<T, kNormChunkBytes> c(tab, blockIdx.x, blocks);
    u32x4 w[kNormWords];
    load_words<STREAM>(c, threadIdx.x, kBlock, w);
    const double all = block_sum<kWaves>(squares(c, threadIdx.x, kBlock, w));
    if (threadIdx.x == 0)
        partial[blockIdx.x] = all;
}

template <int BLOCK>
__global__ __launch_bounds__(BLOCK) void zc_norm_finish_kernel(const double* __restrict__ partial, int64_t blocks,
                                                               float max_norm, float* __restrict__ out)
{
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < blocks; i += 8 * BLOCK) {
        double p[8];                               // eight loads at once, also where fewer are left
#pragma unroll
        for (int c = 0; c < 8; ++c)
            p[c] = partial[i + c * BLOCK < blocks ? i + c * BLOCK : i];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            sum += i + c * BLOCK < blocks ? p[c] : 0.0;
    }
    const double all = block_sum<BLOCK / kLanes>(sum);
    if (threadIdx.x == 0)
        write_norm(all, max_norm, out);
}

// The whole of a short list in one launch, at most two pieces of 8 KB per
// wave, both in flight: 24 tensors of 4 KB take 6 us; two launches take 5.5
// us on the GPU, but 3 us more of the host, which a short list waits for.
template <class T>
__global__ __launch_bounds__(kFinishBlock) void zc_norm_one_kernel(NormTable<kNormShort> tab, uint32_t blocks,
                                                                   float max_norm, float* __restrict__ out)
{
    const int lane = threadIdx.x & (kLanes - 1);
    const uint32_t b = threadIdx.x / kLanes;
    double sum = 0.0;
    if (b < blocks) {
        const uint32_t b2 = b + kFinishWaves;
        const Chunk<T, kPieceBytes> c(tab, b, blocks), d(tab, b2 < blocks ? b2 : b, blocks);
        u32x4 v[kNormWords], w[kNormWords];
        load_words<false>(c, lane, kLanes, v);
        load_words<false>(d, lane, kLanes, w);
        sum = squares(c, lane, kLanes, v);
        sum += b2 < blocks ? squares(d, lane, kLanes, w) : 0.0;
    }
    const double all = block_sum<kFinishWaves>(sum);
    if (threadIdx.x == 0)
        write_norm(all, max_norm, out);
}

// -------------------------------------------------------------------- AdamW

constexpr int kAdamTensors = 52;                   // of a launch, or of a short one (as above)
constexpr int kAdamShort = 16;
constexpr int kAdamRun = 8;                        // values per thread
constexpr int64_t kAdamChunk = kBlock * kAdamRun;
constexpr float kE4m3Max = 448.0f;
constexpr float kE4m3Tiny = 0.001953125f;          // 2^-9, the smallest positive e4m3 value
constexpr float kFlush = 1e-30f;

static_assert(kAdamChunk % ZC_STATE_BLOCK == 0, "whole scale blocks per workgroup");

template <int M>
struct AdamTable {
    zc_adamw_tensor t[M];
    uint32_t first[M];                             // ~0 past the last tensor
};

struct AdamArgs {
    float beta1, rest1, beta2, rest2, eps, keep, rate, root;
};

static_assert(sizeof(AdamTable<kAdamTensors>) + sizeof(AdamArgs) + 8 + 256 <= 4096, "kernel arguments");

// PER e4m3 codes in PER / 4 words, zeros past n.
template <bool STREAM, int PER>
__device__ inline void load_codes(const uint8_t* p, int64_t i, int64_t n, uint32_t (&w)[PER / 4])
{
    if (i + PER <= n) {
        if constexpr (PER == 8) {
            const u32x2 v = load8<STREAM>(p + i);
            w[0] = v[0];
            w[1] = v[1];
        } else {
            w[0] = load4<STREAM>(p + i);
        }
    } else {
#pragma unroll
        for (int h = 0; h < PER / 4; ++h)
            w[h] = 0;
        if (i < n)
#pragma unroll
            for (int c = 0; c < PER; ++c)
                if (i + c < n)
                    w[c / 4] |= static_cast<uint32_t>(p[i + c]) << 8 * (c % 4);
    }
}

template <bool STREAM, int PER>
__device__ inline void store_codes(uint8_t* p, int64_t i, int64_t n, const float (&f)[PER])
{
    uint32_t w[PER / 4];
#pragma unroll
    for (int h = 0; h < PER / 4; ++h) {
        const int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h], f[4 * h + 1], 0, false);
        w[h] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2], f[4 * h + 3], v, true));
    }
    if (i + PER <= n) {
        if constexpr (PER == 8)
            store8<STREAM>(p + i, u32x2{w[0], w[1]});
        else
            store4<STREAM>(p + i, w[0]);
    } else if (i < n) {
#pragma unroll
        for (int c = 0; c < PER; ++c)
            if (i + c < n)
                p[i + c] = static_cast<uint8_t>(w[c / 4] >> 8 * (c % 4));
    }
}

template <int PER>
__device__ inline void decode(const uint32_t (&w)[PER / 4], float scale, float (&f)[PER])
{
#pragma unroll
    for (int h = 0; h < PER / 4; ++h) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], true);
        f[4 * h] = lo[0] * scale;
        f[4 * h + 1] = lo[1] * scale;
        f[4 * h + 2] = hi[0] * scale;
        f[4 * h + 3] = hi[1] * scale;
    }
}

// Largest |x| of the thread's scale block, NaN left out.  (Across the lanes as
// whole numbers: the order of floats that are not negative.)
template <int PER>
__device__ inline float block_top(const float (&f)[PER])
{
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < PER; ++c)
        top = fmaxf(top, fabsf(f[c]));
    return __builtin_bit_cast(float,
                              reduce_max_u32<ZC_STATE_BLOCK / PER>(__builtin_bit_cast(uint32_t, top)));
}

// A workgroup takes 2048 neighbouring values of one tensor, a thread 8 of
// them: every value is read once and written once.  Where a 32-bit array
// takes part, the 8 are two runs of 4, so that a wave's access to it is one
// unbroken kilobyte; else one run of 8 (16 bytes of bf16).
// The states are rounded operation by operation as the definition reads (no
// fused multiply-add, the correctly rounded root), so that another form of the
// same step gives the same 8-bit codes: one unit in the last place of fp32
// would decide a code now and then, and with it the later steps.  So is the
// parameter's step, but for bf16 parameters without masters beside 8-bit
// states (QUICK): there the arithmetic is near the memory's time, and the
// step, which no state follows and which is rounded to bf16, takes fused
// operations and the quotient by the instruction's reciprocal (1 ulp).  90 M
// values with bf16 gradients 158 us so, 163 exact; with masters 252 and 254,
// with fp32 parameters 225 and 228, where the exact one stays.
// Bound by memory: 67 M values with fp32 gradients, masters and states move
// 2.0 GB in 333 us (6.0 TB/s, a copy's rate); 90 M with 8-bit states and bf16
// the rest 0.89 GB in 155 us (5.7), of which the ends of two launches of 52
// tensors take some 5 us.  16 or 32 values per thread: 2 and 15 % slower.
template <class P, class G, bool MASTER, bool E4M3, bool STREAM, int M>
__global__ __launch_bounds__(kBlock) void zc_adamw_kernel(AdamTable<M> tab, AdamArgs a,
                                                          const float* __restrict__ grad_scale)
{
#pragma clang fp contract(off)
    constexpr int PER = sizeof(P) == 2 && sizeof(G) == 2 && !MASTER && E4M3 ? 8 : 4;
    constexpr int RUNS = kAdamRun / PER;
    constexpr bool QUICK = E4M3 && !MASTER && sizeof(P) == 2;
    const float gs = grad_scale ? *grad_scale : 1.0f;
    const int ti = tensor_of(tab.first, blockIdx.x);
    const zc_adamw_tensor t = tab.t[ti];
    const int64_t n = t.n;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x - tab.first[ti]) * kAdamChunk + threadIdx.x * PER;
    P* param = static_cast<P*>(t.param);
    float g[RUNS][PER], m[RUNS][PER], v[RUNS][PER], p[RUNS][PER];
    uint32_t mc[RUNS][PER / 4], vc[RUNS][PER / 4];
    float ms[RUNS], vs[RUNS];
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
        const int64_t i = i0 + r * kBlock * PER;
        load_run<STREAM, PER>(static_cast<const G*>(t.grad), i, n, g[r]);
        if constexpr (MASTER)
            load_run<STREAM, PER>(static_cast<const float*>(t.master), i, n, p[r]);
        else
            load_run<STREAM, PER>(static_cast<const P*>(param), i, n, p[r]);
        if constexpr (E4M3) {
            load_codes<STREAM, PER>(static_cast<const uint8_t*>(t.avg), i, n, mc[r]);
            load_codes<STREAM, PER>(static_cast<const uint8_t*>(t.sq), i, n, vc[r]);
            ms[r] = i < n ? t.avg_scale[i / ZC_STATE_BLOCK] : 0.0f;
            vs[r] = i < n ? t.sq_scale[i / ZC_STATE_BLOCK] : 0.0f;
        } else {
            load_run<STREAM, PER>(static_cast<const float*>(t.avg), i, n, m[r]);
            load_run<STREAM, PER>(static_cast<const float*>(t.sq), i, n, v[r]);
        }
    }
    if (!(fabsf(gs) <= 3.402823466e38f))           // asked for before the loads, looked at after
        return;
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
        const int64_t i = i0 + r * kBlock * PER;
        if constexpr (E4M3) {
            decode<PER>(mc[r], ms[r], m[r]);
            decode<PER>(vc[r], vs[r], v[r]);
#pragma unroll
            for (int c = 0; c < PER; ++c)
                v[r][c] *= v[r][c];
        }
        float q[PER];
#pragma unroll
        for (int c = 0; c < PER; ++c) {
            const float x = g[r][c] * gs;
            m[r][c] = a.beta1 * m[r][c] + a.rest1 * x;
            v[r][c] = a.beta2 * v[r][c] + a.rest2 * (x * x);
            q[c] = sqrtf(v[r][c]);
            if constexpr (QUICK) {
                const float step = m[r][c] * __builtin_amdgcn_rcpf(fmaf(q[c], a.root, a.eps));
                p[r][c] = fmaf(-a.rate, step, p[r][c] * a.keep);
            } else {
                p[r][c] = p[r][c] * a.keep - a.rate * (m[r][c] / (q[c] * a.root + a.eps));
            }
        }
        if constexpr (MASTER)
            store_run<STREAM, PER>(t.master, i, n, p[r]);
        store_run<STREAM, PER>(param, i, n, p[r]);
        if constexpr (E4M3) {
            const float mt = block_top<PER>(m[r]), vt = block_top<PER>(q);
            const bool mk = mt >= kFlush, vk = vt >= kFlush;
            const float mi = mk ? kE4m3Max / mt : 0.0f, vi = vk ? kE4m3Max / vt : 0.0f;
            const float least = vk ? kE4m3Tiny : 0.0f;
#pragma unroll
            for (int c = 0; c < PER; ++c) {
                m[r][c] *= mi;
                const float u = q[c] * vi;
                q[c] = q[c] > 0.0f ? fmaxf(u, least) : u;
            }
            store_codes<STREAM, PER>(static_cast<uint8_t*>(t.avg), i, n, m[r]);
            store_codes<STREAM, PER>(static_cast<uint8_t*>(t.sq), i, n, q);
            if (i < n && i % ZC_STATE_BLOCK == 0) {
                t.avg_scale[i / ZC_STATE_BLOCK] = mk ? mt * (1.0f / kE4m3Max) : 0.0f;
                t.sq_scale[i / ZC_STATE_BLOCK] = vk ? vt * (1.0f / kE4m3Max) : 0.0f;
            }
        } else {
            store_run<STREAM, PER>(static_cast<float*>(t.avg), i, n, m[r]);
            store_run<STREAM, PER>(static_cast<float*>(t.sq), i, n, v[r]);
        }
    }
}

// ---------------------------------------------------------------- launching

int done()
{
    return hipGetLastError() == hipSuccess ? ZC_OK : ZC_EHIP;
}

int64_t chunks(int64_t n, int64_t per)
{
    return (n + per - 1) / per;
}

// Pieces of a list that one workgroup sums alone, 0 for any other.
int64_t norm_pieces(const zc_tensor* tensors, int32_t count, int32_t dtype)
{
    const int64_t bytes = static_cast<int64_t>(elem_bytes(dtype));
    int64_t pieces = 0;
    for (int32_t i = 0; i < count && pieces <= kNormOne; ++i)
        pieces += chunks(tensors[i].n * bytes, kPieceBytes);
    return pieces <= kNormOne ? pieces : 0;
}

// Workgroups of zc_norm_kernel over all tensors, or -1 for a bad argument.
int64_t norm_blocks(const zc_tensor* tensors, int32_t count, int32_t dtype)
{
    if (count < 0 || (count && !tensors) || (dtype != ZC_BF16 && dtype != ZC_F32))
        return -1;
    int64_t all = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (tensors[i].n < 0 || tensors[i].n > (1ll << 48) || (tensors[i].n && !tensors[i].data)
            || misaligned(tensors[i].data, elem_bytes(dtype)))
            return -1;
        all += chunks(tensors[i].n, kNormChunkBytes / static_cast<int64_t>(elem_bytes(dtype)));
    }
    return all <= kMaxBlocks ? all : -1;
}

template <bool B>
struct Bool {
    static constexpr bool value = B;
};

template <class F>
void with_bool(bool b, F f)
{
    if (b)
        f(Bool<true>{});
    else
        f(Bool<false>{});
}

// Calls f with a null pointer of the element type.
template <class F>
void with_type(int32_t dtype, F f)
{
    if (dtype == ZC_BF16)
        f(static_cast<__bf16*>(nullptr));
    else
        f(static_cast<float*>(nullptr));
}

}  // namespace

extern "C" {

size_t zc_grad_norm_workspace_bytes(const zc_tensor* tensors, int32_t count, int32_t dtype)
{
    const int64_t b = norm_blocks(tensors, count, dtype);
    return b <= 0 || norm_pieces(tensors, count, dtype) ? 0 : static_cast<size_t>(b) * sizeof(double);
}

int zc_grad_norm(const zc_tensor* tensors, int32_t count, int32_t dtype, float max_norm, float* d_norm, void* d_ws,
                 size_t ws_bytes, void* stream)
{
    const int64_t blocks = norm_blocks(tensors, count, dtype);
    if (blocks < 0 || !d_norm || misaligned(d_norm, 4) || misaligned(d_ws, 8) || std::isnan(max_norm))
        return ZC_EINVAL;
    const bool one = norm_pieces(tensors, count, dtype) > 0;
    if (!one && blocks && !d_ws)
        return ZC_EINVAL;
    if (!one && ws_bytes < static_cast<size_t>(blocks) * sizeof(double))
        return ZC_ENOSPC;
    hipStream_t s = static_cast<hipStream_t>(stream);
    double* partial = static_cast<double*>(d_ws);
    const int64_t bytes = static_cast<int64_t>(elem_bytes(dtype));
    const bool past = blocks * kNormChunkBytes > kStreamBytes;
    const int64_t per = (one ? kPieceBytes : kNormChunkBytes) / bytes;
    int64_t at = 0;
    const auto launches = [&](auto table, auto launch) {
        constexpr int M = sizeof(table.first) / sizeof(table.first[0]);
        for (int32_t i = 0; i < count;) {
            uint32_t first = 0;
            int m = 0;
            for (; i < count && m < M; ++i) {
                if (tensors[i].n == 0)
                    continue;
                const int64_t c = chunks(tensors[i].n, per);
                table.data[m] = tensors[i].data;
                table.first[m] = first;
                table.last_n[m] = static_cast<uint32_t>(tensors[i].n - (c - 1) * per);
                first += static_cast<uint32_t>(c);
                ++m;
            }
            if (!m)
                break;
            for (int k = m; k < M; ++k) {
                table.data[k] = nullptr;
                table.first[k] = ~0u;
                table.last_n[k] = 0;
            }
            launch(table, first);
            if (hipGetLastError() != hipSuccess)
                return ZC_EHIP;
            at += first;
        }
        return ZC_OK;
    };
    int status = ZC_OK;
    with_type(dtype, [&](auto* type) {
        using T = std::remove_pointer_t<decltype(type)>;
        if (one) {
            status = launches(NormTable<kNormShort>(), [&](const auto& table, uint32_t first) {
                hipLaunchKernelGGL((zc_norm_one_kernel<T>), dim3(1), dim3(kFinishBlock), 0, s, table, first, max_norm,
                                   d_norm);
            });
            return;
        }
        const auto launch = [&](const auto& table, uint32_t first) {
            constexpr int M = sizeof(table.first) / sizeof(table.first[0]);
            if (past)
                hipLaunchKernelGGL((zc_norm_kernel<T, true, M>), dim3(first), dim3(kBlock), 0, s, table, first,
                                   partial + at);
            else
                hipLaunchKernelGGL((zc_norm_kernel<T, false, M>), dim3(first), dim3(kBlock), 0, s, table, first,
                                   partial + at);
        };
        status = count <= kNormShort ? launches(NormTable<kNormShort>(), launch)
                                     : launches(NormTable<kNormTensors>(), launch);
    });
    if (status != ZC_OK)
        return status;
    if (one)
        return ZC_OK;
    if (blocks <= 8 * kLanes)                      // a wave's eight loads per lane
        hipLaunchKernelGGL(zc_norm_finish_kernel<kLanes>, dim3(1), dim3(kLanes), 0, s, partial, blocks, max_norm,
                           d_norm);
    else
        hipLaunchKernelGGL(zc_norm_finish_kernel<kFinishBlock>, dim3(1), dim3(kFinishBlock), 0, s, partial, blocks,
                           max_norm, d_norm);
    return done();
}

int zc_adamw(const zc_adamw_tensor* tensors, int32_t count, const zc_adamw_config* config, const float* d_grad_scale,
             void* stream)
{
    if (count < 0 || (count && !tensors) || !config || misaligned(d_grad_scale, 4))
        return ZC_EINVAL;
    const zc_adamw_config& c = *config;
    const bool e4m3 = c.state_dtype == ZC_E4M3;
    if ((c.param_dtype != ZC_BF16 && c.param_dtype != ZC_F32) || (c.grad_dtype != ZC_BF16 && c.grad_dtype != ZC_F32)
        || (!e4m3 && c.state_dtype != ZC_F32) || c.step < 1 || !(c.beta1 >= 0.0 && c.beta1 < 1.0)
        || !(c.beta2 >= 0.0 && c.beta2 < 1.0) || !(c.eps >= 0.0) || !std::isfinite(c.lr)
        || !std::isfinite(c.weight_decay) || !std::isfinite(c.eps))
        return ZC_EINVAL;
    const size_t pb = elem_bytes(c.param_dtype), gb = elem_bytes(c.grad_dtype), sb = e4m3 ? 1 : 4;
    bool master = false, any = false;
    int64_t all = 0;
    for (int32_t i = 0; i < count; ++i) {
        const zc_adamw_tensor& t = tensors[i];
        if (t.n < 0 || t.n > (1ll << 48))
            return ZC_EINVAL;
        if (t.n == 0)
            continue;
        if (!t.param || !t.grad || !t.avg || !t.sq || (e4m3 && (!t.avg_scale || !t.sq_scale))
            || (any && master != (t.master != nullptr)) || (t.master && c.param_dtype != ZC_BF16))
            return ZC_EINVAL;
        if (misaligned(t.param, pb) || misaligned(t.master, 4) || misaligned(t.grad, gb) || misaligned(t.avg, sb)
            || misaligned(t.sq, sb) || (e4m3 && (misaligned(t.avg_scale, 4) || misaligned(t.sq_scale, 4))))
            return ZC_EINVAL;
        master = t.master != nullptr;
        any = true;
        all += chunks(t.n, kAdamChunk);
    }
    if (all > kMaxBlocks)
        return ZC_EINVAL;

    AdamArgs a;
    a.beta1 = static_cast<float>(c.beta1);
    a.rest1 = static_cast<float>(1.0 - c.beta1);
    a.beta2 = static_cast<float>(c.beta2);
    a.rest2 = static_cast<float>(1.0 - c.beta2);
    a.eps = static_cast<float>(c.eps);
    a.keep = static_cast<float>(1.0 - c.lr * c.weight_decay);
    a.rate = static_cast<float>(c.lr / (1.0 - std::pow(c.beta1, static_cast<double>(c.step))));
    a.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(c.beta2, static_cast<double>(c.step))));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const size_t per = gb + 2 * pb + (master ? 8 : 0) + 4 * sb;
    const bool past = all * kAdamChunk * static_cast<int64_t>(per) > kStreamBytes;
    const auto launches = [&](auto table) {
        constexpr int M = sizeof(table.first) / sizeof(table.first[0]);
        for (int32_t i = 0; i < count;) {
            uint32_t first = 0;
            int m = 0;
            for (; i < count && m < M; ++i) {
                if (tensors[i].n == 0)
                    continue;
                table.t[m] = tensors[i];
                table.first[m] = first;
                first += static_cast<uint32_t>(chunks(tensors[i].n, kAdamChunk));
                ++m;
            }
            if (!m)
                break;
            for (int k = m; k < M; ++k) {
                table.t[k] = zc_adamw_tensor{};
                table.first[k] = ~0u;
            }
            with_type(c.param_dtype, [&](auto* pt) {
                with_type(c.grad_dtype, [&](auto* gt) {
                    with_bool(e4m3, [&](auto e) {
                        with_bool(past, [&](auto x) {
                            using P = std::remove_pointer_t<decltype(pt)>;
                            using G = std::remove_pointer_t<decltype(gt)>;
                            constexpr bool E = decltype(e)::value, X = decltype(x)::value;
                            if (master && sizeof(P) == 2)
                                hipLaunchKernelGGL((zc_adamw_kernel<P, G, sizeof(P) == 2, E, X, M>), dim3(first),
                                                   dim3(kBlock), 0, s, table, a, d_grad_scale);
                            else
                                hipLaunchKernelGGL((zc_adamw_kernel<P, G, false, E, X, M>), dim3(first),
                                                   dim3(kBlock), 0, s, table, a, d_grad_scale);
                        });
                    });
                });
            });
            if (hipGetLastError() != hipSuccess)
                return ZC_EHIP;
        }
        return ZC_OK;
    };
    return count <= kAdamShort ? launches(AdamTable<kAdamShort>()) : launches(AdamTable<kAdamTensors>());
}

}  // extern "C"
