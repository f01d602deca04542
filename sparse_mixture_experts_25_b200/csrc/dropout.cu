// Dropout of the layer's output in front of the residual sum, forward and
// backward, with a mask that is a function of a counter and never stored:
//   m(t, c) = word(t, c) >= rate 2^32
//   forward   out = residual + m Y / (1 - rate)
//   backward  dY  = m dout / (1 - rate)          (d residual = dout)
// word(t, c) is word c mod 4 of Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011) at the 128-bit counter
// (((row0 + t) d + c) / 4, offset) under the 64-bit key `seed`: any kernel, at
// any row of a sharded batch, makes the same mask again.
//
// What bounds it: bytes; 4 + 2 s per element forward and 4 + s backward for an
// s-byte type, read and written once.  A thread has 8 consecutive elements:
// 16-byte accesses, and two generator calls of 20 32-bit products.  A dropped
// element is selected away, not multiplied, so an infinity there leaves 0.
// Measured: 8192 x 4096 bf16 with a residual 40 us (268 MB, 6.7 TB/s), the gradient
// of 8191 x 7168 60 us (352 MB, 5.9 TB/s; the generator keeps the SMs two thirds busy).
#include "moe_internal.cuh"

#include <math.h>

namespace moe {
namespace {

constexpr int kDropThreads = 128;

__device__ __forceinline__ uint4 philox(uint64_t group, uint64_t key, uint64_t offset) {
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

struct DropArgs {
    const void* in;          // Y fp32 (forward) or dout (backward)
    const void* residual;    // forward, nullable
    void* out;
    const uint64_t* step;    // nullable: added to the offset
    uint64_t key, offset;
    int64_t first;           // first group of 4 elements
    int64_t n8;              // groups of 8 elements
    uint32_t threshold;      // words below are dropped
    float scale;
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
// the one rounding to 16 bits: the residual stream's type
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = u;
}

// NONE: rate 0, nothing is drawn.  A thread has U groups of 8 elements, a block's
// width apart, whose loads are on their way while it draws: two where there are
// blocks for several waves (8191 x 7168 gradients 68 -> 63 us), one in small calls
// (17 x 1024 2.3 -> 1.8 us).
template <typename TI, typename TO, bool RESIDUAL, bool NONE, int U>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropArgs a) {
    const int64_t first = (int64_t)blockIdx.x * (kDropThreads * U) + threadIdx.x;
    float v[U][8], out[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * kDropThreads;
        if (i < a.n8) {
            load8(static_cast<const TI*>(a.in) + i * 8, v[u]);
            if (RESIDUAL) load8(static_cast<const TO*>(a.residual) + i * 8, out[u]);
        }
    }
    const uint64_t offset = a.offset + (!NONE && a.step ? *a.step : 0ull);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * kDropThreads;
        if (i >= a.n8) break;
        uint32_t w[8];
        if (!NONE) {
            const uint4 lo = philox((uint64_t)(a.first + 2 * i), a.key, offset);
            const uint4 hi = philox((uint64_t)(a.first + 2 * i + 1), a.key, offset);
            w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
            w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = NONE ? v[u][j] : (w[j] >= a.threshold ? v[u][j] * a.scale : 0.f);
            out[u][j] = RESIDUAL ? out[u][j] + d : d;
        }
        store8(static_cast<TO*>(a.out) + i * 8, out[u]);
    }
}

template <typename TI, typename TO, bool RESIDUAL, int U>
cudaError_t launch_u(const DropArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.n8 + kDropThreads * U - 1) / (kDropThreads * U));
    if (a.threshold) dropout_kernel<TI, TO, RESIDUAL, false, U><<<grid, kDropThreads, 0, st>>>(a);
    else dropout_kernel<TI, TO, RESIDUAL, true, U><<<grid, kDropThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename TI, typename TO, bool RESIDUAL>
cudaError_t launch(const DropArgs& a, cudaStream_t st) {
    // 2048 threads on an SM at once
    return a.n8 >= 4 * 2048 * (int64_t)num_sms() ? launch_u<TI, TO, RESIDUAL, 2>(a, st)
                                                 : launch_u<TI, TO, RESIDUAL, 1>(a, st);
}

moe_status check(const moe_dropout_params* p) {
    if (!p || p->N < 0 || p->d < 1 || p->row0 < 0 || !(p->rate >= 0.0 && p->rate < 1.0)) return MOE_ERR_INVALID_ARG;
    if (p->dtype != MOE_F32 && p->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (p->d % 8) {
        record_error("moe_dropout: d must be a multiple of 8");
        return MOE_ERR_UNSUPPORTED;
    }
    // 2^31 - 1 blocks of at least 2048 elements; element numbers stay below 2^62
    if (p->N > (((int64_t)1 << 42) - 2048) / p->d || p->row0 > ((int64_t)1 << 62) / p->d - p->N) {
        record_error("moe_dropout: N d must be below 2^42 - 2048 and (row0 + N) d at most 2^62");
        return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

DropArgs args_of(const moe_dropout_params& p, const uint64_t* step) {
    DropArgs a{};
    a.step = step;
    a.key = p.seed;
    a.offset = p.offset;
    a.first = p.row0 * p.d / 4;
    a.n8 = p.N * p.d / 8;
    // a rate next to 1 must not wrap to 0: the largest threshold drops all words but one
    a.threshold = (uint32_t)fmin(rint(p.rate * 4294967296.0), 4294967295.0);
    a.scale = (float)(1.0 / (1.0 - p.rate));
    return a;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_dropout_forward(const moe_dropout_params* p, const float* Y, const void* residual, void* out,
                               const uint64_t* step, moe_stream_t stream) {
    const moe_status s = check(p);
    if (s != MOE_OK) return s;
    if (p->N == 0) return MOE_OK;
    if (!Y || !out || !aligned16(Y) || !aligned16(residual) || !aligned16(out) || (reinterpret_cast<uintptr_t>(step) & 7u))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    (void)cudaGetLastError();
    DropArgs a = args_of(*p, step);
    a.in = Y;
    a.residual = residual;
    a.out = out;
    const cudaError_t e = p->dtype == MOE_BF16
                              ? (residual ? launch<float, __nv_bfloat16, true>(a, st) : launch<float, __nv_bfloat16, false>(a, st))
                              : (residual ? launch<float, float, true>(a, st) : launch<float, float, false>(a, st));
    return cuda_status(e, "moe_dropout_forward");
}

moe_status moe_dropout_backward(const moe_dropout_params* p, const void* dout, float* dY, const uint64_t* step,
                                moe_stream_t stream) {
    const moe_status s = check(p);
    if (s != MOE_OK) return s;
    if (p->N == 0) return MOE_OK;
    if (!dout || !dY || !aligned16(dout) || !aligned16(dY) || (reinterpret_cast<uintptr_t>(step) & 7u)) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    (void)cudaGetLastError();
    DropArgs a = args_of(*p, step);
    a.in = dout;
    a.out = dY;
    const cudaError_t e =
        p->dtype == MOE_BF16 ? launch<__nv_bfloat16, float, false>(a, st) : launch<float, float, false>(a, st);
    return cuda_status(e, "moe_dropout_backward");
}

}  // extern "C"
