// The whole sparse-MoE layer for a few tokens (N <= 32), in two launches.
//
// What it computes (the definitions of moe_forward):
//   g = x W_r^T + b, softmax, k largest, weights a, capacity in token order;
//   h = SiLU(x W_g,e^T) (.) (x W_u,e^T);  Y_t = sum_e a_te W_d,e h + shared
//
// What bounds it: each chosen expert's 3 d d_f weights are read once and used
// for a handful of rows, so the floor is those bytes at the copy bandwidth;
// for the smallest layers it is launch and barrier latency.  Hence
//   few_scores_kernel  the router scores as partial sums over K slices (enough
//                      CTAs to read W_r at full rate without a reduction)
//   few_layer_kernel   one CTA per SM, launched cooperatively: every CTA
//                      selects the experts again from the scores (cheaper than
//                      waiting for one CTA to do it), then streams its share
//                      of the gate/up rows, meets the others at one grid
//                      barrier (h is complete), and streams its share of the
//                      down rows.
// The work is cut by weight ROWS, so every CTA reads the same number of bytes
// to within one row whatever the sizes: CTA c of G takes hidden units
// [c T / G, (c+1) T / G) of the T = sum d_f units of the chosen (and shared)
// experts, then output features [c d / G, (c+1) d / G) of every expert.
// A producer warp copies rows with bulk copies into a ring of stages of 16
// rows x 2 KB and runs ahead across tiles, experts and the grid barrier (the
// down weights do not depend on h), so the memory stays busy while the other
// warps reduce and wait.
//
// bf16: mma.sync m16n8k16 with the 16 weight rows as M and the tokens as N;
// the eight consumer warps take K steps of 32 in turn and their partial sums
// meet in shared memory in warp order.  The tensor pipe is nearly idle here:
// a tcgen05 tile (M = 64 or 128 rows) would fix the cut at that many rows and
// leave SMs without work.  A lane reads 8 consecutive K elements of its row
// (16 bytes) and feeds them to two MMAs; both operands use the same order of K,
// so the sum is unchanged.  h is kept as bf16 hi + lo parts (16 mantissa bits,
// relative error 6e-7 rms): rounding it to one bf16 would be the layer's
// largest error, and the second part costs one more MMA on a 1/3 of the bytes.
// fp32: FFMA, one warp per two rows, nothing rounded.
//
// No atomics are used on the outputs: results do not depend on the schedule.
#include "mbarrier.cuh"
#include "moe_internal.cuh"
#include "router_select.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kFewConsumers = 8;                     // consumer warps
constexpr int kFewThreads = 32 * (kFewConsumers + 1);
constexpr int kFewRows = 16;                         // weight rows of a stage
constexpr int kFewChunk = 2048;                      // bytes of a row in a stage
// 64 bytes of padding put two consecutive rows on different halves of the
// banks, so a quarter-warp's 16-byte reads (2 rows x 64 bytes) do not collide
constexpr int kFewPitch = kFewChunk + 64;
constexpr int kFewStage = kFewRows * kFewPitch;
constexpr int kFewMaxPaths = kFewMaxTokens * kMaxK;

struct FewArgs {
    RouterArgs sel;          // selection inputs (ids, w, margin, counters are set by the kernel)
    const void* x;
    const void* W_g;
    const void* W_u;
    const void* W_d;
    const void* Ws_g;
    const void* Ws_u;
    const void* Ws_d;
    const float* part;       // [KS][N][E] partial router scores
    int KS;
    int N, d, d_f, d_sh, E, k;
    int reject;              // moe_reject_policy (zero or renorm)
    int C;                   // requests an expert takes, at most N
    long long C_stat;        // the capacity as the statistics report it
    void* h;                 // bf16: hi plane, lo plane; fp32: one plane.  [N k + N][ldh]
    int64_t h_plane;
    int ldh;
    float* Y;
    unsigned* bar;           // grid barrier, zeroed by the scores kernel
    // records of the routing (workspace)
    int32_t* ids;
    float* w;
    float* margin;
    int32_t* slot;
    int32_t* offsets;
    int32_t* L;
    int32_t* acc;
    int32_t* slot_token;
    float* slot_w;
    float* psum;
    unsigned long long* counters;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two MMAs over the 32 K elements of a step: each lane's 8 elements of its
// rows (lo: row g, hi: row g + 8) against 8 elements of column g
__device__ __forceinline__ void mma_step(float (&c)[4], const uint4& lo, const uint4& hi, const uint4& b) {
    mma_bf16(c, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
    mma_bf16(c, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// ---------------------------------------------------------------------------
// Router scores: CTA (i, q) sums experts 8 i .. 8 i + 7 over K slice q for
// every token, part[q][t][e].  The first CTA also clears the grid barrier and
// the statistics of the call that follows on the stream.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ void __launch_bounds__(256)
    few_scores_kernel(const void* xv, const void* wv, int N, int d, int E, int slice, float* part, unsigned* bar,
                      unsigned long long* counters) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        if (tid == 0) *bar = 0u;
        if (tid < CNT_COUNT) counters[tid] = 0ull;
    }
    const int e0 = blockIdx.x * 8;
    const int k0 = blockIdx.y * slice, k1 = min(d, k0 + slice);
    float* out = part + (int64_t)blockIdx.y * N * E;
    if (BF16) {
        __shared__ float red[8][kFewMaxTokens][9];
        const int g = lane >> 2, t = lane & 3;
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(xv);
        const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(wv);
        const bool two = N > 16;
        float acc[2][4] = {};
        const __nv_bfloat16* wr = e0 + g < E ? w + (int64_t)(e0 + g) * d : nullptr;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        auto ld = [&](const __nv_bfloat16* row, int k, bool ok) {
            return ok ? *reinterpret_cast<const uint4*>(row + k) : zero;
        };
#pragma unroll 2
        for (int k = k0 + warp * 32 + t * 8; k - t * 8 < k1; k += 256) {
            const bool in = k < k1;
            const uint4 b = ld(wr, k, in && wr);
            const uint4 a0 = ld(x + (int64_t)g * d, k, in && g < N);
            const uint4 a1 = ld(x + (int64_t)(g + 8) * d, k, in && g + 8 < N);
            mma_step(acc[0], a0, a1, b);
            if (two) {
                const uint4 a2 = ld(x + (int64_t)(g + 16) * d, k, in && g + 16 < N);
                const uint4 a3 = ld(x + (int64_t)(g + 24) * d, k, in && g + 24 < N);
                mma_step(acc[1], a2, a3, b);
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            red[warp][m * 16 + g][2 * t] = acc[m][0];
            red[warp][m * 16 + g][2 * t + 1] = acc[m][1];
            red[warp][m * 16 + g + 8][2 * t] = acc[m][2];
            red[warp][m * 16 + g + 8][2 * t + 1] = acc[m][3];
        }
        __syncthreads();
        const int tok = tid >> 3, e = e0 + (tid & 7);
        if (tok < N && e < E) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) s += red[q][tok][tid & 7];
            out[(int64_t)tok * E + e] = s;
        }
    } else {
        const float* x = static_cast<const float*>(xv);
        const float* w = static_cast<const float*>(wv);
        const int e = e0 + warp;
        if (e >= E) return;
        const float* wr = w + (int64_t)e * d;
        for (int t0 = 0; t0 < N; t0 += 4) {
            float acc[4] = {};
            for (int k = k0 + lane * 4; k < k1; k += 128) {
                const float4 b = *reinterpret_cast<const float4*>(wr + k);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (t0 + i < N) {
                        const float4 a = *reinterpret_cast<const float4*>(x + (int64_t)(t0 + i) * d + k);
                        acc[i] += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s = warp_sum(acc[i]);
                if (lane == 0 && t0 + i < N) out[(int64_t)(t0 + i) * E + e] = s;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The layer
// ---------------------------------------------------------------------------
struct FewShared {
    int32_t ids[kFewMaxPaths];
    float w[kFewMaxPaths];
    float margin[kFewMaxTokens];
    float psum[kMaxRouterExperts];
    uint32_t asked[kMaxRouterExperts];   // tokens that asked for expert e, one bit each
    uint32_t taken[kMaxRouterExperts];   // tokens it accepted
    int32_t base[kMaxRouterExperts + 1]; // first row of expert e
    int32_t act[kMaxRouterExperts + 1];  // experts with rows, in order
    uint8_t row_tok[kFewMaxPaths];
    float row_w[kFewMaxPaths];
    unsigned long long counters[CNT_COUNT];
    int n_act, n_rows;
    int abort_flag;
};

constexpr int few_stages(int NT) { return NT == 4 ? 4 : 5; }
constexpr size_t few_red_bytes(bool bf16, int NT) { return bf16 ? 2 * 8 * (size_t)NT * 128 * 4 : 0; }
constexpr size_t few_yacc_bytes(bool bf16, int NT) { return (bf16 ? 8 : 1) * (size_t)NT * 8 * kFewRows * 4; }
constexpr size_t few_smem(bool bf16, int NT) {
    return few_stages(NT) * (size_t)kFewStage + few_red_bytes(bf16, NT) + few_yacc_bytes(bf16, NT) + 128 +
           sizeof(FewShared);
}

// a stage position in the ring
struct RingPos {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++stage == n) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// elements of one row that a stage holds: the row in equal pieces of at most
// kFewChunk bytes, multiples of 32 elements
__device__ __forceinline__ int few_chunk(int K, int es) {
    const int n = (int)(((int64_t)K * es + kFewChunk - 1) / kFewChunk);
    return ((K + n - 1) / n + 31) / 32 * 32;
}

// the share [lo, hi) of `total` items of this CTA
__device__ __forceinline__ void few_share(int64_t total, int& lo, int& hi) {
    lo = (int)(total * blockIdx.x / gridDim.x);
    hi = (int)(total * (blockIdx.x + 1) / gridDim.x);
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <bool BF16, int NT>
__global__ void __launch_bounds__(kFewThreads, 1) few_layer_kernel(const __grid_constant__ FewArgs a) {
    constexpr int ST = few_stages(NT);
    constexpr int ES = BF16 ? 2 : 4;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    float* red = reinterpret_cast<float*>(smem + ST * kFewStage);
    float* yacc = reinterpret_cast<float*>(smem + ST * kFewStage + few_red_bytes(BF16, NT));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + ST * kFewStage + few_red_bytes(BF16, NT) +
                                                 few_yacc_bytes(BF16, NT));
    uint64_t* empty = full + ST;
    FewShared& S = *reinterpret_cast<FewShared*>(reinterpret_cast<uint8_t*>(full) + 128);
    static_assert(2 * ST * 8 <= 128, "barriers");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort_flag = &S.abort_flag;

    // ---- routing: every CTA selects all tokens' experts ----
    for (int i = tid; i < kMaxRouterExperts; i += kFewThreads) {
        S.asked[i] = 0u;
        S.psum[i] = 0.f;
    }
    if (tid < CNT_COUNT) S.counters[tid] = 0ull;
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kFewConsumers);
        }
        S.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    {
        RouterArgs r = a.sel;
        r.ids = S.ids;
        r.w = S.w;
        r.margin = S.margin;
        r.counters = S.counters;
        float* ps = blockIdx.x == 0 ? S.psum : nullptr;  // only one CTA writes the records
        auto load = [&](int t, int e) {
            if (e >= a.E) return -INFINITY;
            float s = 0.f;
            for (int q = 0; q < a.KS; ++q) s += a.part[((int64_t)q * a.N + t) * a.E + e];
            return a.sel.b_r ? s + a.sel.b_r[e] : s;
        };
        for (int t = warp; t < a.N; t += kFewConsumers + 1) {
            if (a.E <= 32) {
                float v[1] = {load(t, lane)};
                select_token<1>(r, t, lane, v, ps);
            } else if (a.E <= 128) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = load(t, lane + 32 * i);
                select_token<4>(r, t, lane, v, ps);
            } else {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = load(t, lane + 32 * i);
                select_token<8>(r, t, lane, v, ps);
            }
        }
    }
    __syncthreads();
    const int paths = a.N * a.k;
    for (int i = tid; i < paths; i += kFewThreads)
        if (S.ids[i] >= 0) atomicOr(&S.asked[S.ids[i]], 1u << (i / a.k));
    __syncthreads();
    for (int e = tid; e < a.E; e += kFewThreads) {
        uint32_t m = S.asked[e];
        for (int over = __popc(m) - a.C; over > 0; --over) m &= ~(0x80000000u >> __clz(m));  // the first C stay
        S.taken[e] = m;
    }
    __syncthreads();
    if (warp == 0) {
        int rows = 0, n = 0;
        for (int b = 0; b < a.E; b += 32) {
            const int e = b + lane;
            const int c = e < a.E ? __popc(S.taken[e]) : 0;
            int v = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (e < a.E) S.base[e] = rows + v - c;
            const unsigned have = __ballot_sync(0xffffffffu, c > 0);
            if (c > 0) S.act[n + __popc(have & ((1u << lane) - 1u))] = e;
            rows += __shfl_sync(0xffffffffu, v, 31);
            n += __popc(have);
        }
        if (lane == 0) {
            S.base[a.E] = rows;
            S.n_rows = rows;
            S.n_act = n;
        }
    }
    __syncthreads();
    for (int i = tid; i < paths; i += kFewThreads) {
        const int e = S.ids[i], t = i / a.k;
        if (e < 0 || !((S.taken[e] >> t) & 1u)) continue;
        const int r = S.base[e] + __popc(S.taken[e] & ((1u << t) - 1u));
        float wc = S.w[i];
        if (a.reject == MOE_REJECT_RENORM) {  // a token that lost a path shares its weight out again
            float sum = 0.f;
            bool lost = false;
            for (int j = t * a.k; j < (t + 1) * a.k; ++j) {
                const int f = S.ids[j];
                if (f < 0) continue;
                if ((S.taken[f] >> t) & 1u) sum += S.w[j];
                else lost = true;
            }
            if (lost && sum > 0.f) wc = wc / sum;
        }
        S.row_tok[r] = (uint8_t)t;
        S.row_w[r] = wc;
    }
    __syncthreads();

    const int n_act = S.n_act, n_rows = S.n_rows;
    const int n_groups = n_act + (a.d_sh > 0 ? 1 : 0);
    int u0, u1, c0, c1;
    few_share((int64_t)n_act * a.d_f + a.d_sh, u0, u1);
    few_share(a.d, c0, c1);
    // tile at unit u: the group, its first unit, and how many (at most 8, inside the group and the share)
    auto unit_tile = [&](int u, int& gi, int& j, int& nj) {
        gi = u < n_act * a.d_f ? u / a.d_f : n_act;
        j = u - gi * a.d_f;
        nj = min(min(8, (gi < n_act ? a.d_f : a.d_sh) - j), u1 - u);
    };

    if (warp == kFewConsumers) {
        // ---- producer ----
        RingPos pos;
        int used = 0;  // stages filled at least once
        bool ok = true;
        auto fill = [&](int rows, const uint8_t* src, uint32_t bytes, int row_slot) {
            // lanes 0 .. rows - 1 copy their row; src is this lane's
            if (!warp_wait_bounded(&empty[pos.stage], pos.phase ^ 1u, abort_flag, a.counters)) return false;
            if (lane == 0) mbar_expect_tx(&full[pos.stage], rows * bytes);
            __syncwarp();
            if (lane < rows)
                bulk_load(smem_u32(ring) + pos.stage * kFewStage + row_slot * kFewPitch, src, bytes,
                          &full[pos.stage]);
            if (used < ST) ++used;
            pos.next(ST);
            return true;
        };
        const int lenA = few_chunk(a.d, ES);
        for (int u = u0; u < u1 && ok;) {
            int gi, j, nj;
            unit_tile(u, gi, j, nj);
            const bool up = lane >= nj;
            const int jj = j + (up ? lane - nj : lane);
            const uint8_t* W = static_cast<const uint8_t*>(gi < n_act ? (up ? a.W_u : a.W_g) : (up ? a.Ws_u : a.Ws_g));
            const int64_t row = (gi < n_act ? (int64_t)S.act[gi] * a.d_f : 0) + jj;
            const uint8_t* src = W + row * a.d * ES;
            for (int kb = 0; kb < a.d && ok; kb += lenA)
                ok = fill(2 * nj, src + (int64_t)kb * ES, (uint32_t)(min(lenA, a.d - kb) * ES), up ? 8 + lane - nj : lane);
            u += nj;
        }
        for (int c = c0; c < c1 && ok; c += kFewRows) {
            const int nc = min(kFewRows, c1 - c);
            for (int gi = 0; gi < n_groups && ok; ++gi) {
                const int K = gi < n_act ? a.d_f : a.d_sh;
                const int len = few_chunk(K, ES);
                const uint8_t* W = static_cast<const uint8_t*>(gi < n_act ? a.W_d : a.Ws_d);
                const int64_t row = (gi < n_act ? (int64_t)S.act[gi] * a.d : 0) + c + lane;
                const uint8_t* src = W + row * K * ES;
                for (int kb = 0; kb < K && ok; kb += len)
                    ok = fill(nc, src + (int64_t)kb * ES, (uint32_t)(min(len, K - kb) * ES), lane);
            }
        }
        // every copy has landed before the CTA may leave, also when a wait
        // gave up: the last fill of each used stage, with a limit
        const unsigned long long t0 = global_timer_ns();
        for (int s = 0; s < used; ++s) {
            const uint32_t par = s < pos.stage ? pos.phase : pos.phase ^ 1u;
            while (!mbar_try_wait(smem_u32(&full[s]), par) && global_timer_ns() - t0 < kTimeoutNs) {
            }
        }
    } else {
        // ---- consumers ----
        RingPos pos;
        const int g = lane >> 2, t = lane & 3;
        const uint4 zero4 = make_uint4(0, 0, 0, 0);
        // bf16: one group's rows (16 weight rows against `ntr` column tiles),
        // summed over K; `ptr` the columns' rows (null: no such column)
        auto mma_rows = [&](int K, const __nv_bfloat16* const (&ptr)[NT], int planes, int64_t plane, int ntr,
                            float (&acc)[NT][4]) {
            constexpr int PF = NT == 1 ? 4 : (NT == 2 ? 2 : 1);
            const int len0 = few_chunk(K, 2);
            for (int kb = 0; kb < K; kb += len0) {
                const int len = min(len0, K - kb);
                const int steps = (len + 31) / 32;
                const uint8_t* st = ring + pos.stage * kFewStage;
                bool waited = false, ok = true;
                for (int s0 = warp; s0 < steps || !waited; s0 += kFewConsumers * PF) {
                    // the columns' operands first: their latency passes while the rows arrive
                    uint4 b[PF][2][NT];
#pragma unroll
                    for (int p = 0; p < PF; ++p) {
                        const int kk = (s0 + p * kFewConsumers) * 32 + t * 8;
#pragma unroll
                        for (int pl = 0; pl < 2; ++pl)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                b[p][pl][n] = (kk < len && ptr[n] && pl < planes)
                                                  ? *reinterpret_cast<const uint4*>(ptr[n] + pl * plane + kb + kk)
                                                  : zero4;
                    }
                    if (!waited) {
                        ok = warp_wait_bounded(&full[pos.stage], pos.phase, abort_flag, a.counters);
                        waited = true;
                    }
                    if (!ok) break;
#pragma unroll
                    for (int p = 0; p < PF; ++p) {
                        const int s = s0 + p * kFewConsumers;
                        if (s >= steps) break;
                        const int kk = s * 32 + t * 8;
                        uint4 lo = zero4, hi = zero4;
                        if (kk < len) {  // what lies behind a row's end in the stage is not a number to use
                            lo = *reinterpret_cast<const uint4*>(st + g * kFewPitch + kk * 2);
                            hi = *reinterpret_cast<const uint4*>(st + (g + 8) * kFewPitch + kk * 2);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (n < ntr) {
                                mma_step(acc[n], lo, hi, b[p][0][n]);
                                if (planes > 1) mma_step(acc[n], lo, hi, b[p][1][n]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[pos.stage]);
                pos.next(ST);
            }
        };
        // fp32: rows `warp` and `warp + 8` of the stage against R columns
        auto ffma_rows = [&](int K, const float* x, int64_t ldx, const uint8_t* tok, int R, float (&acc)[2][NT * 8]) {
            const int len0 = few_chunk(K, 4);
            for (int kb = 0; kb < K; kb += len0) {
                const int len = min(len0, K - kb);
                const uint8_t* st = ring + pos.stage * kFewStage;
                if (warp_wait_bounded(&full[pos.stage], pos.phase, abort_flag, a.counters)) {
                    for (int kk = lane * 4; kk < len; kk += 128) {
                        const float4 p = *reinterpret_cast<const float4*>(st + warp * kFewPitch + kk * 4);
                        const float4 q = *reinterpret_cast<const float4*>(st + (warp + 8) * kFewPitch + kk * 4);
#pragma unroll
                        for (int r = 0; r < NT * 8; ++r) {
                            if (r < R) {
                                const int row = tok ? tok[r] : r;
                                const float4 v = *reinterpret_cast<const float4*>(x + row * ldx + kb + kk);
                                acc[0][r] += p.x * v.x + p.y * v.y + p.z * v.z + p.w * v.w;
                                acc[1][r] += q.x * v.x + q.y * v.y + q.z * v.z + q.w * v.w;
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[pos.stage]);
                pos.next(ST);
            }
        };

        // gate/up: h of this CTA's hidden units
        int tile = 0;
        for (int u = u0; u < u1; ++tile) {
            int gi, j, nj;
            unit_tile(u, gi, j, nj);
            const bool routed = gi < n_act;
            const int e = routed ? S.act[gi] : 0;
            const int row0 = routed ? S.base[e] : n_rows;
            const int R = routed ? __popc(S.taken[e]) : a.N;
            const uint8_t* tok = routed ? S.row_tok + row0 : nullptr;
            if constexpr (BF16) {
                const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
                const __nv_bfloat16* ptr[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int r = n * 8 + g;
                    ptr[n] = r < R ? x + (int64_t)(tok ? tok[r] : r) * a.d : nullptr;
                }
                float acc[NT][4] = {};
                const int ntr = (R + 7) / 8;
                mma_rows(a.d, ptr, 1, 0, ntr, acc);
                // warps' partial sums: [n][16 rows][8 columns], two buffers in turn
                float* mine = red + ((tile & 1) * 8 + warp) * (NT * 128);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    *reinterpret_cast<float2*>(mine + n * 128 + g * 8 + 2 * t) = make_float2(acc[n][0], acc[n][1]);
                    *reinterpret_cast<float2*>(mine + n * 128 + (g + 8) * 8 + 2 * t) = make_float2(acc[n][2], acc[n][3]);
                }
                consumer_sync();
                const int unit = tid & 7, r = tid >> 3;
                if (r < R && unit < nj) {
                    const float* p = red + (tile & 1) * 8 * (NT * 128) + (r >> 3) * 128 + unit * 8 + (r & 7);
                    float zg = 0.f, zu = 0.f;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        zg += p[q * (NT * 128)];
                        zu += p[q * (NT * 128) + 64];
                    }
                    const float hv = zg / (1.0f + expf(-zg)) * zu;
                    const __nv_bfloat16 hi = __float2bfloat16_rn(hv);
                    __nv_bfloat16* h = static_cast<__nv_bfloat16*>(a.h) + (int64_t)(row0 + r) * a.ldh + j + unit;
                    h[0] = hi;
                    // an infinite h has no second part
                    const float rest = hv - __bfloat162float(hi);
                    h[a.h_plane] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
                }
            } else {
                float acc[2][NT * 8] = {};
                ffma_rows(a.d, static_cast<const float*>(a.x), a.d, tok, R, acc);
#pragma unroll
                for (int r = 0; r < NT * 8; ++r) {
                    if (r < R) {
                        const float zg = warp_sum(acc[0][r]), zu = warp_sum(acc[1][r]);
                        if (lane == (r & 31) && warp < nj)
                            static_cast<float*>(a.h)[(int64_t)(row0 + r) * a.ldh + j + warp] =
                                zg / (1.0f + expf(-zg)) * zu;
                    }
                }
            }
            u += nj;
        }

        // grid barrier: every CTA's part of h is written
        __threadfence();
        consumer_sync();
        if (tid == 0) {
            atomicAdd(a.bar, 1u);
            const unsigned long long t0 = global_timer_ns();
            for (uint32_t it = 1;; ++it) {
                unsigned seen;
                asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(a.bar) : "memory");
                if (seen >= gridDim.x) break;
                if ((it & 63u) == 0) {
                    if (*abort_flag) break;
                    if (global_timer_ns() - t0 > kTimeoutNs) {
                        *abort_flag = 1;
                        atomicOr(a.counters + CNT_DEVICE_ERROR, (unsigned long long)DEVERR_TIMEOUT);
                        break;
                    }
                }
            }
        }
        consumer_sync();
        __threadfence();

        // down: this CTA's output features, summed over the experts in order
        for (int c = c0; c < c1; c += kFewRows) {
            const int nc = min(kFewRows, c1 - c);
            for (int i = tid; i < (BF16 ? 8 : 1) * NT * 8 * kFewRows; i += 256) yacc[i] = 0.f;
            consumer_sync();
            for (int gi = 0; gi < n_groups; ++gi) {
                const bool routed = gi < n_act;
                const int e = routed ? S.act[gi] : 0;
                const int row0 = routed ? S.base[e] : n_rows;
                const int R = routed ? __popc(S.taken[e]) : a.N;
                const int K = routed ? a.d_f : a.d_sh;
                if constexpr (BF16) {
                    const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(a.h);
                    const __nv_bfloat16* ptr[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int r = n * 8 + g;
                        ptr[n] = r < R ? h + (int64_t)(row0 + r) * a.ldh : nullptr;
                    }
                    float acc[NT][4] = {};
                    mma_rows(K, ptr, 2, a.h_plane, (R + 7) / 8, acc);
                    // into this warp's sums [token][16 features]: a token has one row in a group
                    float* mine = yacc + warp * (NT * 8 * kFewRows);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = n * 8 + 2 * t + i;
                            if (r < R) {
                                const int tk = routed ? S.row_tok[row0 + r] : r;
                                const float wt = routed ? S.row_w[row0 + r] : 1.f;
                                mine[tk * kFewRows + g] += wt * acc[n][i];
                                mine[tk * kFewRows + g + 8] += wt * acc[n][2 + i];
                            }
                        }
                    __syncwarp();
                } else {
                    float acc[2][NT * 8] = {};
                    ffma_rows(K, static_cast<const float*>(a.h) + (int64_t)row0 * a.ldh, a.ldh, nullptr, R, acc);
#pragma unroll
                    for (int r = 0; r < NT * 8; ++r) {
                        if (r < R) {
                            const float s0 = warp_sum(acc[0][r]), s1 = warp_sum(acc[1][r]);
                            if (lane == 0) {  // features `warp` and `warp + 8` belong to this warp
                                const int tk = routed ? S.row_tok[row0 + r] : r;
                                const float wt = routed ? S.row_w[row0 + r] : 1.f;
                                yacc[tk * kFewRows + warp] += wt * s0;
                                yacc[tk * kFewRows + warp + 8] += wt * s1;
                            }
                        }
                    }
                }
            }
            consumer_sync();
            for (int i = tid; i < a.N * kFewRows; i += 256) {
                const int tk = i / kFewRows, f = i % kFewRows;
                if (f >= nc) continue;
                float s = 0.f;
#pragma unroll
                for (int q = 0; q < (BF16 ? 8 : 1); ++q) s += yacc[q * (NT * 8 * kFewRows) + i];
                a.Y[(int64_t)tk * a.d + c + f] = s;
            }
            consumer_sync();
        }

        // routing records and statistics, by the first CTA, after its share of the layer
        if (blockIdx.x == 0) {
            for (int i = tid; i < paths; i += 256) {
                const int e = S.ids[i], tk = i / a.k;
                const bool in = e >= 0 && ((S.taken[e] >> tk) & 1u);
                a.ids[i] = e;
                a.w[i] = S.w[i];
                a.slot[i] = in ? __popc(S.taken[e] & ((1u << tk) - 1u)) : -1;
            }
            for (int i = tid; i < n_rows; i += 256) {
                a.slot_token[i] = S.row_tok[i];
                a.slot_w[i] = S.row_w[i];
            }
            for (int e = tid; e <= a.E; e += 256) {
                a.offsets[e] = S.base[e];
                if (e < a.E) {
                    a.L[e] = __popc(S.asked[e]);
                    a.acc[e] = __popc(S.taken[e]);
                    a.psum[e] = S.psum[e];
                }
            }
            if (tid < a.N) a.margin[tid] = S.margin[tid];
            if (warp == 0) {
                int req = 0, over = 0, top = 0, affected = 0, skipped = 0;
                for (int e = lane; e < a.E; e += 32) {
                    const int l = __popc(S.asked[e]);
                    req += l;
                    over += (int)max(0ll, l - a.C_stat);
                    top = max(top, l);
                }
                if (lane < a.N) {
                    int asked = 0, got = 0;
                    for (int j = lane * a.k; j < (lane + 1) * a.k; ++j) {
                        const int e = S.ids[j];
                        if (e < 0) continue;
                        ++asked;
                        got += (S.taken[e] >> lane) & 1u;
                    }
                    affected = got < asked;
                    skipped = asked > 0 && got == 0;
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    req += __shfl_xor_sync(0xffffffffu, req, o);
                    over += __shfl_xor_sync(0xffffffffu, over, o);
                    affected += __shfl_xor_sync(0xffffffffu, affected, o);
                    skipped += __shfl_xor_sync(0xffffffffu, skipped, o);
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                }
                if (lane == 0) {
                    a.counters[CNT_REQUESTED] = req;
                    a.counters[CNT_ACCEPTED] = n_rows;
                    a.counters[CNT_REJECTED] = req - n_rows;
                    a.counters[CNT_O] = over;
                    a.counters[CNT_AFFECTED] = affected;
                    a.counters[CNT_SKIPPED] = skipped;
                    a.counters[CNT_NONFINITE] = S.counters[CNT_NONFINITE];
                    a.counters[CNT_NEAR_TIE] = S.counters[CNT_NEAR_TIE];
                    a.counters[CNT_L_MAX] = top;
                    a.counters[CNT_C] = a.C_stat;
                }
            }
        }
    }
    __syncthreads();
}

// K slices of the router scores: about one CTA per SM, at least 256 elements
// (a step of every warp) each
int few_score_slices(int d, int E) {
    const int blocks = (E + 7) / 8;
    return std::max(1, std::min(std::min(16, num_sms() / blocks), d / 256));
}

template <bool BF16, int NT>
cudaError_t launch_layer(const FewArgs& a, cudaStream_t st) {
    auto kern = few_layer_kernel<BF16, NT>;
    const size_t smem = few_smem(BF16, NT);
    static_assert(few_smem(BF16, NT) <= 232448, "shared memory per CTA");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)num_sms(), 1, 1);
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    // all CTAs are resident together: they meet at a grid barrier
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

FewLayout few_layout(const moe_params& p, size_t after) {
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    FewLayout L;
    L.bar = after;
    L.part = L.bar + 256;
    L.h = L.part + up((size_t)few_score_slices(p.d, p.E_r) * p.N * p.E_r * 4);
    const size_t rows = (size_t)p.N * p.k + (p.d_f_shared > 0 ? (size_t)p.N : 0);
    L.total = L.h + up(rows * (size_t)std::max(p.d_f, p.d_f_shared) * 4);
    return L;
}

cudaError_t launch_few(const moe_params& p, int64_t C, const void* x, const void* W_r, const float* b_r,
                       const float* lat, const ExpertWeights& W, float* Y, const WsView& v, const FewLayout& L,
                       cudaStream_t st) {
    const bool bf16 = p.dtype == MOE_BF16;
    const int KS = few_score_slices(p.d, p.E_r);
    const int slice = ((p.d + KS - 1) / KS + 31) / 32 * 32;
    FewArgs a{};
    a.sel.b_r = b_r;
    a.sel.lat = lat;
    a.sel.N = p.N;
    a.sel.d = p.d;
    a.sel.E = p.E_r;
    a.sel.k = p.k;
    a.sel.norm = p.norm;
    a.sel.theta = p.theta;
    a.x = x;
    a.W_g = W.W_g;
    a.W_u = W.W_u;
    a.W_d = W.W_d;
    a.Ws_g = W.Ws_g;
    a.Ws_u = W.Ws_u;
    a.Ws_d = W.Ws_d;
    float* part = reinterpret_cast<float*>(v.base + L.part);
    a.part = part;
    a.KS = KS;
    a.N = (int)p.N;
    a.d = p.d;
    a.d_f = p.d_f;
    a.d_sh = p.d_f_shared;
    a.E = p.E_r;
    a.k = p.k;
    a.reject = p.reject_policy;
    a.C = (int)min64(C, p.N);
    a.C_stat = C;
    a.h = v.base + L.h;
    a.ldh = std::max(p.d_f, p.d_f_shared);
    a.h_plane = ((int64_t)p.N * p.k + (p.d_f_shared > 0 ? p.N : 0)) * a.ldh;
    a.Y = Y;
    a.bar = reinterpret_cast<unsigned*>(v.base + L.bar);
    a.ids = v.ids;
    a.w = v.w;
    a.margin = v.margin;
    a.slot = v.slot;
    a.offsets = v.offsets;
    a.L = v.L;
    a.acc = v.acc;
    a.slot_token = v.slot_token;
    a.slot_w = v.slot_w;
    a.psum = v.scratch.psum;
    a.counters = v.counters;
    const dim3 grid((unsigned)((p.E_r + 7) / 8), (unsigned)KS);
    if (bf16) few_scores_kernel<true><<<grid, 256, 0, st>>>(x, W_r, a.N, p.d, p.E_r, slice, part, a.bar, v.counters);
    else few_scores_kernel<false><<<grid, 256, 0, st>>>(x, W_r, a.N, p.d, p.E_r, slice, part, a.bar, v.counters);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (bf16) {
        if (p.N <= 8) return launch_layer<true, 1>(a, st);
        if (p.N <= 16) return launch_layer<true, 2>(a, st);
        return launch_layer<true, 4>(a, st);
    }
    if (p.N <= 8) return launch_layer<false, 1>(a, st);
    if (p.N <= 16) return launch_layer<false, 2>(a, st);
    return launch_layer<false, 4>(a, st);
}

}  // namespace moe
