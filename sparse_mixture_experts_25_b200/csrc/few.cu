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
// The work is cut by weight ROWS, so the CTAs finish together whatever the
// sizes: CTA c of G takes its share of the hidden units of all chosen (and
// shared) experts, each weighted by what its expert's stages cost, then output
// features [c d / G, (c+1) d / G) of every expert.
// Producer warps copy pieces of 16 weight rows (down: of up to 32), and of the
// tokens' rows that they meet, into a ring of stages with bulk copies; a piece is
// as long as a stage has room for, 1 to 3 KB where there are few tokens.  They
// run ahead across tiles and experts, and fill the ring with down weights
// before the grid barrier (only the rows of h wait for it), so the memory stays
// busy while the other warps reduce and wait.  There are four of them because a
// warp takes about 32 ns to issue a copy: on rings that are only emptied, 16
// rows of 1 KB a stage reach 4.0 TB/s with one producer warp, 6.2 with two and
// 7.3 with four.
//
// bf16: mma.sync m16n8k16 with the 16 weight rows as M and the tokens as N;
// the eight consumer warps take K steps of 32 in turn and their partial sums
// meet in shared memory in warp order.  The tensor pipe is nearly idle here
// (7% of its cycles for one token of 8 chosen experts of 4096 x 1536):
// a tcgen05 tile (M = 64 or 128 rows) would fix the cut at that many rows and
// leave SMs without work.  A lane reads 8 consecutive K elements of its row
// (16 bytes) and feeds them to two MMAs; both operands use the same order of K,
// so the sum is unchanged.  h is kept as three bf16 parts (24 mantissa bits):
// rounding it to one bf16 would be the layer's largest error by far, two parts
// still left Y 2.5e-6 of its norm off, and the third costs one more MMA on a
// third of the bytes.
// fp32: FFMA, a warp per eight weight rows and up to eight tokens, nothing rounded.
//
// Measured (both launches, replayed from a graph): one token through 8 of 128
// experts of 4096 x 1536 61 us, 4.9 TB/s (the two kernels, the barrier and the
// first stages are 10 us of that); 7 tokens of 6 to 8 experts of 4096 x 14336 377
// us and 32 tokens of 165 of 256 experts of 7168 x 2048 2190 us, both above the
// 6.55 TB/s of a copy; one fp32 token of a 256 x 512 expert 13.3 us, all latency.
//
// No atomics are used on the outputs: results do not depend on the schedule.
#include "mbarrier.cuh"
#include "moe_internal.cuh"
#include "router_select.cuh"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

constexpr int kFewConsumers = 8;                     // consumer warps
constexpr int kFewProducers = 4;                     // producer warps
constexpr int kFewThreads = 32 * (kFewConsumers + kFewProducers);
constexpr int kFewRows = 16;                         // weight rows of a stage
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
    uint8_t* h;              // hidden activations, laid out as the down stages take them (few_h)
    int h_row;               // bytes set aside for a row
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

// two MMAs over the 32 K elements of a step: each lane's 8 elements of its
// rows (lo: row g, hi: row g + 8) against 8 elements of column g.  They sum
// into two accumulators, so that neither waits for the other
__device__ __forceinline__ void mma_step(float (&c)[4], float (&d)[4], const uint4& lo, const uint4& hi,
                                         const uint4& b) {
    mma_bf16(c, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
    mma_bf16(d, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
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
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the layer's CTAs may get ready
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
        float acc[4][4] = {};
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
            mma_step(acc[0], acc[2], a0, a1, b);
            if (two) {
                const uint4 a2 = ld(x + (int64_t)(g + 16) * d, k, in && g + 16 < N);
                const uint4 a3 = ld(x + (int64_t)(g + 24) * d, k, in && g + 24 < N);
                mma_step(acc[1], acc[3], a2, a3, b);
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            red[warp][m * 16 + g][2 * t] = acc[m][0] + acc[m + 2][0];
            red[warp][m * 16 + g][2 * t + 1] = acc[m][1] + acc[m + 2][1];
            red[warp][m * 16 + g + 8][2 * t] = acc[m][2] + acc[m + 2][2];
            red[warp][m * 16 + g + 8][2 * t + 1] = acc[m][3] + acc[m + 2][3];
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
// An expert with rows (or the shared one, last): its weight matrices' row
// block, its rows of h, and how its rows are cut into stages
struct FewGroup {
    int e;               // expert, 0 for the shared one
    int row0, R;         // first row (h, row_tok, row_w) and number of rows
    int F;               // hidden units
    int len1, pitch1;    // gate/up pieces (rows of d)
    int len2, pitch2;    // down pieces (rows of F)
    int hrow;            // bytes of a row of h in a down piece
    int unit_cost;       // relative cost of a gate/up unit
};

struct FewShared {
    int32_t ids[kFewMaxPaths];
    float w[kFewMaxPaths];
    float margin[kFewMaxTokens];
    float psum[kMaxRouterExperts];
    uint32_t asked[kMaxRouterExperts];   // tokens that asked for expert e, one bit each
    uint32_t taken[kMaxRouterExperts];   // tokens it accepted
    int32_t base[kMaxRouterExperts + 1]; // first row of expert e
    FewGroup grp[kMaxRouterExperts + 1]; // experts with rows, in order, then the shared one
    uint32_t cost[kMaxRouterExperts + 2]; // cost of the gate/up units of the groups before
    uint8_t row_tok[kFewMaxPaths];
    float row_w[kFewMaxPaths];
    unsigned long long counters[CNT_COUNT];
    int warp_rows[8], warp_n[8];         // rows and experts with rows among each 32 experts
    int from[2], to[2];                  // this CTA's units: group and unit, from and to
    int abort_flag;
};

// stages of the ring and their size: the rest of the shared memory holds the
// reductions, which grow with the token tiles NT
// (three large stages beat four of 3/4 the size, 32 tokens of 128 experts 803 ->
// 751 us, and five or six of 2/3 lose)
constexpr int kFewStages = 3;
constexpr int few_stage_bytes(int NT) { return NT == 1 ? 61 * 1024 : (NT == 2 ? 58 * 1024 : 53 * 1024); }
// gate/up: partial sums of 8 warps, two buffers; down: 8 warps' sums per token
constexpr int few_down_rows(bool bf16) { return bf16 ? 2 * kFewRows : kFewRows; }
constexpr size_t few_red_bytes(int NT) { return 2 * 8 * 128 * 4 * (size_t)NT; }
static_assert(few_red_bytes(1) >= 8 * 8 * few_down_rows(true) * 4, "the down sums fit where the gate/up ones were");
constexpr size_t few_smem(int NT) {
    return kFewStages * (size_t)few_stage_bytes(NT) + few_red_bytes(NT) + 128 + sizeof(FewShared);
}

// column tiles of a form for a group's rows (few_layer_kernel's by_rows); 0 stands for one, packed
template <int M>
__device__ __forceinline__ constexpr int column_tiles(std::integral_constant<int, M>) {
    return M ? M : 1;
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

// How rows of K elements are cut: `len` elements a piece (equal pieces, multiples
// of 32 elements, at most what `rows` weight rows and R other rows of `parts`
// pieces each leave room for), weight rows `pitch` bytes apart.  The pitch is 64 bytes
// above a multiple of 128, which puts two consecutive rows on different halves of
// the banks, so a quarter-warp's 16-byte reads (2 rows x 64 bytes) do not collide.
__device__ __forceinline__ void few_cut(int K, int es, int rows, int R, int parts, int stage_bytes, int& len, int& pitch) {
    const int room = (stage_bytes - (rows + R) * 64) / (rows + R * parts);
    const int cap = (room & ~127) / es;  // elements, a multiple of 32
    const int n = (K + cap - 1) / cap;
    len = ((K + n - 1) / n + 31) / 32 * 32;
    pitch = cap * es + 64;
}

// Bytes of a row of h in a down piece: its parts one after another, and 64 more
// where that is a multiple of 128.  A group's h is stored piece by piece, each
// with all rows of the group, so that a stage takes its rows of h in one copy.
__device__ __forceinline__ int few_h_row(int len, int es, int parts) {
    const int bytes = len * es * parts;
    return bytes % 128 ? bytes : bytes + 64;
}
// more than a row of h can take over all its pieces of at least 64 elements
inline size_t few_h_bound(int F, int es, int parts) {
    return ((size_t)F * es * parts + (size_t)(F / 64 + 1) * (32 * es * parts + 64) + 127) / 128 * 128;
}

// Sums each of N values over the warp's lanes, halving what a lane holds at each
// step: lane i is left with the sums of values i N / 32 and on, in v[0], v[1] ...
template <int N, int LEFT = N / 2, int FROM = 16>
__device__ __forceinline__ void lane_sums(float (&v)[N], int lane) {
    const bool high = lane & FROM;
#pragma unroll
    for (int i = 0; i < LEFT; ++i) {
        const float theirs = high ? v[i] : v[i + LEFT], mine = high ? v[i + LEFT] : v[i];
        v[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, FROM);
    }
    if constexpr (FROM > 1) lane_sums<N, LEFT / 2, FROM / 2>(v, lane);
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <bool BF16, int NT>
__global__ void __launch_bounds__(kFewThreads, 1) few_layer_kernel(const __grid_constant__ FewArgs a) {
    constexpr int ST = kFewStages;
    constexpr int SB = few_stage_bytes(NT);
    constexpr int ES = BF16 ? 2 : 4;
    constexpr int PL = BF16 ? 3 : 1;  // parts that h is kept in
    constexpr int DR = few_down_rows(BF16);  // weight rows of a down stage
    static_assert((SB - (DR + NT * 8) * 64) / (DR + PL * NT * 8) >= (BF16 ? 128 : 256),
                  "a stage holds at least 64 elements of every row");
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    float* red = reinterpret_cast<float*>(smem + ST * SB);
    float* yacc = red;  // gate/up is over when the down sums begin
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + ST * SB + few_red_bytes(NT));
    uint64_t* empty = full + ST;
    uint64_t* h_ready = empty + ST;
    FewShared& S = *reinterpret_cast<FewShared*>(reinterpret_cast<uint8_t*>(full) + 128);
    static_assert((2 * ST + 1) * 8 <= 128, "barriers");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort_flag = &S.abort_flag;
    // the output features of a CTA go in equal tiles of at most DR, as many in every
    // CTA: h is cut into pieces for their size
    const int c_most = (a.d + gridDim.x - 1) / gridDim.x, c_tiles = (c_most + DR - 1) / DR;
    const int c_rows = (c_most + c_tiles - 1) / c_tiles;

    // ---- routing: every CTA selects all tokens' experts ----
    for (int i = tid; i < kMaxRouterExperts; i += kFewThreads) {
        S.asked[i] = 0u;
        S.psum[i] = 0.f;
    }
    if (tid < CNT_COUNT) S.counters[tid] = 0ull;
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], kFewProducers);
            mbar_init(&empty[s], kFewConsumers);
        }
        mbar_init(h_ready, 1);
        S.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // launched while the scores kernel runs: its results count from here on
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    {
        RouterArgs r = a.sel;
        r.ids = S.ids;
        r.w = S.w;
        r.margin = S.margin;
        r.counters = S.counters;
        float* ps = blockIdx.x == 0 ? S.psum : nullptr;  // only one CTA writes the records
        // scores: the K slices' sums in order, in the ring's memory
        float* g = reinterpret_cast<float*>(ring);
        const int ne = a.N * a.E;
        if (a.E % 4 == 0) {
#pragma unroll 2
            for (int i = tid * 4; i < ne; i += kFewThreads * 4) {
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int q = 0; q < a.KS; ++q) {
                    const float4 v = *reinterpret_cast<const float4*>(a.part + (int64_t)q * ne + i);
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
                *reinterpret_cast<float4*>(g + i) = s;
            }
        } else {
            for (int i = tid; i < ne; i += kFewThreads) {
                float s = 0.f;
#pragma unroll 4
                for (int q = 0; q < a.KS; ++q) s += a.part[(int64_t)q * ne + i];
                g[i] = s;
            }
        }
        __syncthreads();
        auto load = [&](int t, int e) {
            return e < a.E ? g[t * a.E + e] + (a.sel.b_r ? a.sel.b_r[e] : 0.f) : -INFINITY;
        };
        for (int t = warp; t < a.N; t += kFewThreads / 32) {
            if (a.E <= 32) {
                float v[1] = {load(t, lane)};
                select_token<1>(r, t, lane, v, ps);
            } else {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = load(t, lane + 32 * i);
                select_token<8>(r, t, lane, v, ps);
            }
        }
    }
    fence_async_smem();  // the ring's memory is the copies' from here on
    __syncthreads();
    const int paths = a.N * a.k;
    for (int i = tid; i < paths; i += kFewThreads)
        if (S.ids[i] >= 0) atomicOr(&S.asked[S.ids[i]], 1u << (i / a.k));
    __syncthreads();
    // accepted tokens, rows and groups: a warp for every 32 experts
    int e_rows = 0, e_at = 0, e_n = 0;
    unsigned e_have = 0;
    if (warp < 8) {
        const int e = tid;
        uint32_t m = e < a.E ? S.asked[e] : 0u;
        for (int over = __popc(m) - a.C; over > 0; --over) m &= ~(0x80000000u >> __clz(m));  // the first C stay
        if (e < a.E) S.taken[e] = m;
        e_rows = __popc(m);
        e_at = e_rows;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, e_at, o);
            if (lane >= o) e_at += u;
        }
        e_have = __ballot_sync(0xffffffffu, e_rows > 0);
        if (lane == 31) S.warp_rows[warp] = e_at;
        if (lane == 0) S.warp_n[warp] = __popc(e_have);
        e_at -= e_rows;
    }
    __syncthreads();
    int n_rows = 0, n_act = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        if (q == warp) {
            e_at += n_rows;
            e_n = n_act;
        }
        n_rows += S.warp_rows[q];
        n_act += S.warp_n[q];
    }
    const int n_groups = n_act + (a.d_sh > 0 ? 1 : 0);
    if (warp < 8 && tid < a.E) S.base[tid] = e_at;
    const bool own = warp < 8 && e_rows > 0, shared = tid == kFewThreads - 1 && a.d_sh > 0;
    if (own || shared) {
        FewGroup gr;
        gr.e = own ? tid : 0;
        gr.row0 = own ? e_at : n_rows;
        gr.R = own ? e_rows : a.N;
        gr.F = own ? a.d_f : a.d_sh;
        few_cut(a.d, ES, kFewRows, gr.R, 1, SB, gr.len1, gr.pitch1);
        few_cut(gr.F, ES, c_rows, gr.R, PL, SB, gr.len2, gr.pitch2);
        gr.hrow = few_h_row(gr.len2, ES, PL);
        // a unit's cost: its stages' bytes at an SM's share of the memory (47
        // bytes/ns) or the issue of their copies (18 ns each), whichever is
        // longer, in 1/16 of the first (at most 255)
        const int n = (a.d + gr.len1 - 1) / gr.len1;
        const int mem = a.d * (kFewRows * ES) / 47 + 1, issue = n * (kFewRows + gr.R) * 18;
        gr.unit_cost = issue > mem ? min(255, (int)(issue * 16ll / mem)) : 16;
        const int at = own ? e_n + __popc(e_have & ((1u << lane) - 1u)) : n_act;
        S.grp[at] = gr;
        S.cost[at + 1] = (uint32_t)gr.unit_cost * gr.F;
    }
    if (tid == 0) {
        S.base[a.E] = n_rows;
        S.cost[0] = 0;
    }
    __syncthreads();
    if (warp == 0) {
        // this CTA's share of the gate/up units, as a span of (group, unit)
        uint32_t sum = 0;
        for (int b = 0; b < n_groups; b += 32) {
            const int i = b + lane;
            uint32_t v = i < n_groups ? S.cost[i + 1] : 0u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (i < n_groups) S.cost[i + 1] = sum + v;
            sum += __shfl_sync(0xffffffffu, v, 31);
        }
        __syncwarp();
        if (lane < 2) {
            const uint32_t c = blockIdx.x + lane, q = sum / gridDim.x, at = q * c + (sum - q * gridDim.x) * c / gridDim.x;
            int lo = 0, hi = n_groups;  // the last group that begins at or before `at` (n_groups at the end)
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (S.cost[mid] <= at) lo = mid;
                else hi = mid - 1;
            }
            int* out = lane ? S.to : S.from;
            out[0] = lo;
            out[1] = lo < n_groups ? (int)((at - S.cost[lo]) / (uint32_t)S.grp[lo].unit_cost) : 0;
        }
    } else {
        for (int i = tid - 32; i < paths; i += kFewThreads - 32) {
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
    }
    __syncthreads();
    const int g_to = S.to[0], j_to = S.to[1];
    // the next tile of at most 8 units of a group, from (gi, j) on; false at the end of the share
    auto unit_tile = [&](int& gi, int& j, int& nj) {
        if (gi < n_groups && j >= S.grp[gi].F) {
            ++gi;
            j = 0;
        }
        if (gi > g_to || (gi == g_to && j >= j_to)) return false;
        nj = min(8, (gi == g_to ? j_to : S.grp[gi].F) - j);
        return true;
    };
    const int c0 = (int)((int64_t)a.d * blockIdx.x / gridDim.x), c1 = (int)((int64_t)a.d * (blockIdx.x + 1) / gridDim.x);

    if (warp >= kFewConsumers) {
        // ---- producers: row i of a stage is copied by lane i / 4 of warp i % 4 ----
        const int mine = lane * kFewProducers + warp - kFewConsumers;
        static_assert(kFewRows + kFewMaxTokens <= 32 * kFewProducers && DR + 1 <= 32 * kFewProducers, "a lane for every row of a stage");
        RingPos pos;
        int used = 0;  // stages filled at least once
        // takes the next stage, which this warp copies its share of `rows` pieces of `bytes`, and `more`, to
        auto open = [&](int rows, uint32_t bytes, uint32_t more) {
            if (!warp_wait_bounded(&empty[pos.stage], pos.phase ^ 1u, abort_flag, a.counters)) return false;
            if (lane == 0)
                mbar_expect_tx(&full[pos.stage],
                               (rows + kFewProducers - 1 - (warp - kFewConsumers)) / kFewProducers * bytes + more);
            __syncwarp();
            if (used < ST) ++used;
            return true;
        };
        auto copy = [&](int stage, int slot, int pitch, const uint8_t* src, uint32_t bytes) {
            bulk_load(smem_u32(ring) + stage * SB + slot * pitch, src, bytes, &full[stage]);
        };
        auto gate_up = [&]() {
            int nj;
            for (int gi = S.from[0], j = S.from[1]; unit_tile(gi, j, nj); j += nj) {
                const FewGroup gr = S.grp[gi];
                const int rows = 2 * nj + gr.R;
                // this lane's row: a gate row, an up row or a token's row
                const uint8_t* src = nullptr;
                int slot = 0;
                if (mine < 2 * nj) {
                    const bool up = mine >= nj;
                    const int jj = up ? mine - nj : mine;
                    const void* m = gi < n_act ? (up ? a.W_u : a.W_g) : (up ? a.Ws_u : a.Ws_g);
                    src = static_cast<const uint8_t*>(m) + ((int64_t)gr.e * a.d_f + j + jj) * a.d * ES;
                    slot = (up ? 8 : 0) + jj;
                } else if (mine < rows) {
                    const int r = mine - 2 * nj;
                    const int tok = gi < n_act ? S.row_tok[gr.row0 + r] : r;
                    src = static_cast<const uint8_t*>(a.x) + (int64_t)tok * a.d * ES;
                    slot = kFewRows + r;
                }
                for (int kb = 0; kb < a.d; kb += gr.len1) {
                    const uint32_t bytes = (uint32_t)(min(gr.len1, a.d - kb) * ES);
                    if (!open(rows, bytes, 0)) return false;
                    if (src) copy(pos.stage, slot, gr.pitch1, src + (int64_t)kb * ES, bytes);
                    pos.next(ST);
                }
            }
            return true;
        };
        // the down stages in order.  Those before `skip` are passed over; of the
        // next `count`, `weights` opens the stage and copies the weight rows,
        // `rows` copies the rows of h into it (without weights: into the stages from `at` on)
        auto down = [&](int skip, int count, bool weights, bool rows, RingPos at) {
            int n = 0;
            for (int c = c0; c < c1; c += c_rows) {
                const int nc = min(c_rows, c1 - c);
                for (int gi = 0; gi < n_groups; ++gi) {
                    const FewGroup gr = S.grp[gi];
                    // weight rows as above; the rows of h, one copy, by the lane after the last of them
                    const bool mine_w = mine < nc, mine_h = mine == nc;
                    const uint8_t* src = static_cast<const uint8_t*>(gi < n_act ? a.W_d : a.Ws_d) +
                                         ((int64_t)gr.e * a.d + c + mine) * gr.F * ES;
                    const uint32_t h_bytes = (uint32_t)(gr.R * gr.hrow);
                    const uint8_t* hsrc = a.h + (int64_t)gr.row0 * a.h_row;
                    const uint32_t mine_more = nc % kFewProducers == warp - kFewConsumers ? h_bytes : 0;
                    for (int kb = 0; kb < gr.F; kb += gr.len2, ++n, hsrc += h_bytes) {
                        if (n < skip) continue;
                        if (n >= skip + count) return true;
                        const uint32_t bytes = (uint32_t)(min(gr.len2, gr.F - kb) * ES);
                        if (weights) {
                            if (!open(nc, bytes, mine_more)) return false;
                            at = pos;
                            pos.next(ST);
                            if (mine_w) copy(at.stage, mine, gr.pitch2, src + (int64_t)kb * ES, bytes);
                        }
                        if (rows && mine_h) copy(at.stage, c_rows, gr.pitch2, hsrc, h_bytes);
                        if (!weights) at.next(ST);
                    }
                }
            }
            return true;
        };
        bool ok = gate_up();
        if (ok) {
            // a ring full of down weights, then (h is complete) their rows of h, then the rest
            const RingPos first = pos;
            ok = down(0, ST, true, false, pos) && warp_wait_bounded(h_ready, 0u, abort_flag, a.counters);
            if (ok) {
                // h was written by ordinary stores, of all CTAs; the copies read it
                asm volatile("fence.proxy.async;" ::: "memory");
                ok = down(0, ST, false, true, first) && down(ST, 0x7fffffff - ST, true, true, pos);
            }
        }
        // routing records and statistics, by the first CTA's producers, which are done
        // before the consumers are
        if (blockIdx.x == 0) {
            const int ptid = tid - 32 * kFewConsumers;
            for (int i = ptid; i < paths; i += 32 * kFewProducers) {
                const int e = S.ids[i], tk = i / a.k;
                const bool in = e >= 0 && ((S.taken[e] >> tk) & 1u);
                a.ids[i] = e;
                a.w[i] = S.w[i];
                a.slot[i] = in ? __popc(S.taken[e] & ((1u << tk) - 1u)) : -1;
            }
            for (int i = ptid; i < n_rows; i += 32 * kFewProducers) {
                a.slot_token[i] = S.row_tok[i];
                a.slot_w[i] = S.row_w[i];
            }
            for (int e = ptid; e <= a.E; e += 32 * kFewProducers) {
                a.offsets[e] = S.base[e];
                if (e < a.E) {
                    a.L[e] = __popc(S.asked[e]);
                    a.acc[e] = __popc(S.taken[e]);
                    a.psum[e] = S.psum[e];
                }
            }
            if (ptid < a.N) a.margin[ptid] = S.margin[ptid];
            if (ptid < 32) {
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
        // bf16: a stage's `rows` weight rows (WT tiles of 16) against a group's R token
        // rows (`planes` parts each), summed over K: the warps take the steps of 32 in
        // turn.  (The tensor pipe truncates its running sums, so a piece's products
        // are summed from zero and added to the sum outside, with rounding: left to
        // run over K, Y was off by 2.5e-6 of its norm, ten times as much.)
        auto mma_rows = [&](auto row_tiles, auto tiles, int rows, int K, int piece, int pitch, int R, int row_bytes, auto planes,
                            float (&sum)[decltype(row_tiles)::value][column_tiles(decltype(tiles){})][4]) {
            // M column tiles of 8, or (0) the three parts of one or two rows as the
            // columns of one tile: part q of row r is column 2 q + r
            constexpr int WT = decltype(row_tiles)::value, M = column_tiles(tiles);
            constexpr bool PACKED = decltype(tiles)::value == 0;
            constexpr int P = PACKED ? 1 : decltype(planes)::value;
            constexpr int CH = P > 1 && WT * M <= 2 ? 4 : 2;  // accumulators in turn: more hide more latency
            for (int kb = 0; kb < K; kb += piece) {
                const int len = min(piece, K - kb);
                float acc[CH][WT][M][4] = {};
                const uint8_t* st = ring + pos.stage * SB;
                if (warp_wait_bounded(&full[pos.stage], pos.phase, abort_flag, a.counters)) {
#pragma unroll WT * M == 1 ? 4 : 2
                    for (int kk = warp * 32 + t * 8; kk - t * 8 < len; kk += 32 * kFewConsumers) {
                        const bool in = kk < len;  // what lies behind a row's end in the stage is not a number to use
                        const uint8_t* col = st + kk * 2;
                        auto ld = [&](const uint8_t* p, bool have) {
                            return have && in ? *reinterpret_cast<const uint4*>(p) : zero4;
                        };
                        uint4 lo[WT], hi[WT];
#pragma unroll
                        for (int w = 0; w < WT; ++w) {
                            lo[w] = ld(col + (w * 16 + g) * pitch, w * 16 + g < rows);
                            hi[w] = ld(col + (w * 16 + g + 8) * pitch, w * 16 + g + 8 < rows);
                        }
#pragma unroll
                        for (int n = 0; n < M; ++n) {
                            if (M == 1 || n * 8 < R) {
                                const bool have = PACKED ? (g & 1) < R && g < 6 : n * 8 + g < R;
                                const uint8_t* row = col + rows * pitch +
                                                     (PACKED ? (g & 1) * row_bytes + (g >> 1) * 2 * piece
                                                             : (n * 8 + g) * row_bytes);
#pragma unroll
                                for (int q = P - 1; q >= 0; --q) {  // small parts first
                                    const uint4 b = ld(row + 2 * q * piece, have);
#pragma unroll
                                    for (int w = 0; w < WT; ++w)
                                        mma_step(acc[q ? CH - 2 : 0][w][n], acc[q ? CH - 1 : 1][w][n], lo[w], hi[w], b);
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[pos.stage]);
                pos.next(ST);
#pragma unroll
                for (int w = 0; w < WT; ++w)
#pragma unroll
                    for (int n = 0; n < M; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            sum[w][n][i] += acc[0][w][n][i] + acc[1][w][n][i];
                            if (CH == 4) sum[w][n][i] += acc[CH - 2][w][n][i] + acc[CH - 1][w][n][i];
                        }
            }
        };
        // fp32: a stage's `rows` weight rows against R token rows.  A warp has 8 of the
        // weight rows, T (4 or 8) of the tokens and every KP-th step of 64 of K, so that
        // a value from shared memory meets T or 8 others.  acc[8 r + i]: token r, weight
        // row i, summed over this lane's part of K.  A row or token past the last is
        // taken for the last one, and its sums are not used.  (Two weight rows and all
        // tokens a warp waited for shared memory: 18 experts of 136 x 6200 and 11 tokens
        // 564 us instead of 192 to 206, 19 of 4600 x 80 and 18 tokens 128 instead of 52.
        // At 32 rows the sums still bound it: 2 experts of 7168 x 7168 take 828 us, 4.4
        // times their bytes.)
        struct Part {
            int rg, tg, kp, KP;  // which rows, tokens and steps of K
        };
        auto token_groups = [](int R) { return R > 16 ? 4 : R > 8 ? 2 : 1; };
        auto part_of = [&](int rows, int R) {
            const int RG = rows > 8 ? 2 : 1, TG = token_groups(R);
            return Part{warp & (RG - 1), warp / RG & (TG - 1), warp / (RG * TG), kFewConsumers / (RG * TG)};
        };
        auto ffma_rows = [&](auto tokens, int rows, int K, int piece, int pitch, int R, int row_bytes,
                             float (&acc)[decltype(tokens)::value * 8]) __attribute__((always_inline)) {
            constexpr int T = decltype(tokens)::value;
            const Part me = part_of(rows, R);
            const bool mine = me.tg * 8 < R;
            const int row_last = rows - 1 - me.rg * 8, tok_last = R - 1 - me.tg * 8;
            int w_at[8], x_at[T];
#pragma unroll
            for (int i = 0; i < 8; ++i) w_at[i] = (me.rg * 8 + min(i, row_last)) * pitch + lane * 8;
#pragma unroll
            for (int r = 0; r < T; ++r) x_at[r] = rows * pitch + (me.tg * 8 + min(r, tok_last)) * row_bytes + lane * 8;
            for (int kb = 0; kb < K; kb += piece) {
                const int len = min(piece, K - kb);
                const uint8_t* st = ring + pos.stage * SB;
                if (warp_wait_bounded(&full[pos.stage], pos.phase, abort_flag, a.counters) && mine) {
                    auto step = [&](int kk) __attribute__((always_inline)) {
                        const uint8_t* at = st + kk * 4;
                        float2 p[8], v[T];
#pragma unroll
                        for (int i = 0; i < 8; ++i) p[i] = *reinterpret_cast<const float2*>(at + w_at[i]);
#pragma unroll
                        for (int r = 0; r < T; ++r) v[r] = *reinterpret_cast<const float2*>(at + x_at[r]);
#pragma unroll
                        for (int r = 0; r < T; ++r)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                acc[r * 8 + i] = fmaf(p[i].x, v[r].x, acc[r * 8 + i]);
#pragma unroll
                        for (int r = 0; r < T; ++r)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                acc[r * 8 + i] = fmaf(p[i].y, v[r].y, acc[r * 8 + i]);
                    };
                    int kk = me.kp * 64;
#pragma unroll 1
                    for (; kk + 64 <= len; kk += me.KP * 64) step(kk);
                    if (kk + lane * 2 < len) step(kk);  // the last, short one
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[pos.stage]);
                pos.next(ST);
            }
        };
        auto by_tokens = [&](int R, auto f) {
            if (R <= 4) f(std::integral_constant<int, 4>{});
            else f(std::integral_constant<int, 8>{});
        };

        // the form for a group's rows: as many column tiles as they fill (a
        // group of a few rows in a batch of 32 tokens needs one, not four)
        auto by_rows = [&](int R, auto f) {
            if (NT > 1 && R <= 8) f(std::integral_constant<int, 1>{});
            else if (NT > 2 && R <= 16) f(std::integral_constant<int, 2>{});
            else f(std::integral_constant<int, NT>{});
        };
        const std::integral_constant<int, 1> x_parts{};
        const std::integral_constant<int, PL> h_parts{};
        const std::integral_constant<int, 1> unit_tiles{};
        const std::integral_constant<int, DR / 16> down_tiles{};

        // gate/up: h of this CTA's hidden units
        int tile = 0, nj;
        for (int gi = S.from[0], j = S.from[1]; unit_tile(gi, j, nj); j += nj, ++tile) {
            const FewGroup gr = S.grp[gi];
            const int R = gr.R;
            // where h of row r and unit j goes: its piece, the row in it, the unit in that
            auto h_at = [&](int r, int unit) {
                const int piece = unit / gr.len2;
                return a.h + (int64_t)gr.row0 * a.h_row + ((int64_t)piece * R + r) * gr.hrow + (unit - piece * gr.len2) * ES;
            };
            if constexpr (BF16) {
                // warps' partial sums: [n][16 rows][8 columns], two buffers in turn
                float* mine = red + ((tile & 1) * 8 + warp) * (NT * 128);
                by_rows(R, [&](auto tiles) {
                    constexpr int M = decltype(tiles)::value;
                    float sum[1][M][4] = {};
                    mma_rows(unit_tiles, tiles, kFewRows, a.d, gr.len1, gr.pitch1, R, gr.pitch1, x_parts, sum);
#pragma unroll
                    for (int n = 0; n < M; ++n) {
                        const float(&c)[4] = sum[0][n];
                        *reinterpret_cast<float2*>(mine + n * 128 + g * 8 + 2 * t) = make_float2(c[0], c[1]);
                        *reinterpret_cast<float2*>(mine + n * 128 + (g + 8) * 8 + 2 * t) = make_float2(c[2], c[3]);
                    }
                });
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
                    float hv = zg / (1.0f + expf(-zg)) * zu;
                    __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(h_at(r, j + unit));
#pragma unroll
                    for (int q = 0; q < PL; ++q) {
                        // the first part is cut off: rounded, the largest finite h would be infinite
                        const __nv_bfloat16 part = q ? __float2bfloat16_rn(hv) : __float2bfloat16_rz(hv);
                        h[q * gr.len2] = part;
                        hv -= __bfloat162float(part);
                        hv = isfinite(hv) ? hv : 0.f;  // one that is not finite is its first part
                    }
                }
            } else {
                // warps' partial sums (those that have a step of K): [tokens][8 rows], two buffers in turn
                float* mine = red + ((tile & 1) * 8 + warp) * (NT * 128);
                const Part me = part_of(kFewRows, R);
                const int len = min(gr.len1, a.d);
                by_tokens(R, [&](auto tokens) {
                    constexpr int T = decltype(tokens)::value;
                    float acc[T * 8] = {};
                    ffma_rows(tokens, kFewRows, a.d, gr.len1, gr.pitch1, R, gr.pitch1, acc);
                    if (me.kp * 64 < len) {
                        lane_sums(acc, lane);
#pragma unroll
                        for (int i = 0; i < T / 4; ++i) mine[lane * (T / 4) + i] = acc[i];
                    }
                });
                consumer_sync();
                const int unit = tid & 7, r = tid >> 3;
                if (r < R && unit < nj) {
                    const int TG = token_groups(R);
                    const float* p = red + ((tile & 1) * 8 + (r >> 3) * 2) * (NT * 128) + (r & 7) * 8 + unit;
                    float zg = 0.f, zu = 0.f;
                    for (int q = 0; q < kFewConsumers && q / (2 * TG) * 64 < len; q += 2 * TG) {
                        zg += p[q * (NT * 128)];
                        zu += p[(q + 1) * (NT * 128)];
                    }
                    *reinterpret_cast<float*>(h_at(r, j + unit)) = zg / (1.0f + expf(-zg)) * zu;
                }
            }
        }

        // grid barrier: every CTA's part of h is written, also for the copies that will read it
        asm volatile("fence.proxy.async;" ::: "memory");
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
        if (tid == 0) mbar_arrive(h_ready);

        // down: this CTA's output features, summed over the experts in order
        for (int c = c0; c < c1; c += c_rows) {
            const int nc = min(c_rows, c1 - c);
            for (int i = tid; i < 8 * NT * 8 * DR; i += 256) yacc[i] = 0.f;
            consumer_sync();
            for (int gi = 0; gi < n_groups; ++gi) {
                const bool routed = gi < n_act;
                const FewGroup gr = S.grp[gi];
                const int row0 = gr.row0, R = gr.R;
                // into this warp's sums [token][DR features]: a token has one row in a group
                float* mine = yacc + warp * (NT * 8 * DR);
                if constexpr (BF16) {
                    const auto add = [&](auto tiles) {
                        constexpr int M = column_tiles(tiles);
                        float sum[DR / 16][M][4] = {};
                        mma_rows(down_tiles, tiles, c_rows, gr.F, gr.len2, gr.pitch2, R, gr.hrow, h_parts, sum);
                        if (decltype(tiles)::value == 0) {  // the parts' columns, small ones first, in the lanes of part 0
#pragma unroll
                            for (int w = 0; w < DR / 16; ++w)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    float& v = sum[w][0][i];
                                    const float mid = __shfl_down_sync(0xffffffffu, v, 1);
                                    v += __shfl_down_sync(0xffffffffu, v, 2) + mid;
                                }
                        }
#pragma unroll
                        for (int n = 0; n < M; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int r = n * 8 + 2 * t + i;
                                if (r < R) {
                                    const int tk = routed ? S.row_tok[row0 + r] : r;
                                    const float wt = routed ? S.row_w[row0 + r] : 1.f;
#pragma unroll
                                    for (int w = 0; w < DR / 16; ++w) {
                                        mine[tk * DR + w * 16 + g] += wt * sum[w][n][i];
                                        mine[tk * DR + w * 16 + g + 8] += wt * sum[w][n][2 + i];
                                    }
                                }
                            }
                    };
                    // one or two rows (a layer of many experts, or one token): all parts in one MMA
                    if (R <= 2) add(std::integral_constant<int, 0>{});
                    else by_rows(R, add);
                    __syncwarp();
                } else {
                    const Part me = part_of(c_rows, R);
                    by_tokens(R, [&](auto tokens) {
                        constexpr int T = decltype(tokens)::value;
                        float acc[T * 8] = {};
                        ffma_rows(tokens, c_rows, gr.F, gr.len2, gr.pitch2, R, gr.hrow, acc);
                        if (me.kp * 64 >= min(gr.len2, gr.F)) return;  // no step of K
                        lane_sums(acc, lane);
#pragma unroll
                        for (int i = 0; i < T / 4; ++i) {
                            const int at = lane * (T / 4) + i, r = me.tg * 8 + at / 8, f = me.rg * 8 + at % 8;
                            if (r < R && f < c_rows) {
                                const int tk = routed ? S.row_tok[row0 + r] : r;
                                mine[tk * DR + f] += (routed ? S.row_w[row0 + r] : 1.f) * acc[i];
                            }
                        }
                    });
                    __syncwarp();
                }
            }
            consumer_sync();
            for (int i = tid; i < a.N * DR; i += 256) {
                const int tk = i / DR, f = i % DR;
                if (f >= nc) continue;
                float s = 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q) s += yacc[q * (NT * 8 * DR) + i];
                a.Y[(int64_t)tk * a.d + c + f] = s;
            }
            consumer_sync();
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
    const size_t smem = few_smem(NT);
    static_assert(few_smem(NT) <= 232448, "shared memory per CTA");
    cudaError_t e = allow_smem_once<few_layer_kernel<BF16, NT>>(smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)num_sms(), 1, 1);
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    // all CTAs are resident together: they meet at a grid barrier.  They are
    // set up while the scores kernel runs
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
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
    L.h_row = few_h_bound(std::max(p.d_f, p.d_f_shared), (int)esize(p.dtype), p.dtype == MOE_BF16 ? 3 : 1);
    L.total = L.h + up(rows * L.h_row);
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
    a.h = reinterpret_cast<uint8_t*>(v.base + L.h);
    a.h_row = (int)L.h_row;
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
