// Low-rank adapters of many requests at once, beside a shared projection or
// beside the whole layer, with their gradients.
//
// Token t has adapter a = ids[t] (or none).  With u_t = s_a A_a x_t and
// v_t = s_a B_a^T dy_t (both r numbers):
//   forward    y_t  = base_t + W x_t + B_a u_t
//   backward   dx_t = base_t + W^T dy_t + A_a^T v_t
//              dA_a = sum_t v_t x_t^T,  dB_a = sum_t dy_t u_t^T
// over the tokens of adapter a.
//
// What bounds them: r is 8 to 128 while the widths are thousands, so each step
// reads one [N, width] array and writes another or none; the floor is those
// bytes.  Three kinds of kernel, each one pass over its wide array:
//   shrink  [N, K] x [K, r]  -> u or v        reads x or dy
//   expand  [N, r] x [r, J]  -> y or dx       reads base, writes y or dx
//   grad    [r, n] x [n, J]  -> dA or dB      reads x or dy over a's tokens
// A stable counting sort (plan) puts the tokens of an adapter next to one
// another, so a tile of 64 rows has one adapter and reads it once; the rows are
// gathered and scattered where they are used, not copied.  The sort is stable
// and nothing is summed by atomics: results do not depend on the schedule.
//
// Arithmetic: mma.sync m16n8k16 on bf16 parts, fp32 accumulation.  A 16-bit
// operand is one part; a 32-bit one is the sum of three bf16 parts (24 bits), and
// where two of them meet the products of parts up to 2^-16 of the first are kept
// (six of nine).  With two parts (16 bits) the results were 2.5e-6 to 4.6e-6 of
// their norm off.  (tcgen05 tiles of 64 or 128 rows
// would be mostly padding at these ranks: the tensor pipe is not what bounds.)
// u and v are stored as such parts, in the sorted order.  The tensor pipe
// truncates its running sums: left to run over K = 1000 in fp32, y was off by
// 4.9e-6 of its norm.  So a long sum is kept outside: the products of up to four
// stages (256 K of a shrink, 128 tokens of a gradient; a stage's small parts
// first) are summed from zero and added to it with rounding.
//
// Few tokens take another form (see takes_tokens): no sort, one CTA per token
// and slice of K, then one thread per output; two launches instead of three, and
// no row of a tile is wasted on a token with an adapter of its own.
//
// The kernels of a call are set up while the one before runs and wait for it
// themselves (programmatic launches), which saves about half a microsecond each.
//
// W runs on the layer's own GEMMs (tcgen05 for bf16, dy as two bf16 parts): its
// sums run over all of K in the tensor pipe, which truncates them, so y is 4.4e-6 of
// its norm off at K = 4096 and dx 5.0e-6 (1.5e-6 and 2.9e-6 at 1536; 1e-6 or less
// without W).  Two parts of dy are a choice: their 16 bits are 2.4e-6 of that, added
// at right angles, and a third would take half of that GEMM's time again (26 us of
// 118, 2047 tokens, 4096 to 1536).
//
// Measured, replayed from a graph: 16 tokens with 16 adapters (d = 4096, r = 16) 5
// us; 4096 tokens of 32 adapters through a 4096 x 4096 projection 141 to 155 us, 101
// of them the projection; gradients of 8192 tokens of four adapters (d = 4096, r =
// 64) 280 to 350 us by how many of the tokens have an adapter, of which the products
// of parts, 69 GFLOP on mma.sync at about 550 TFLOP/s, are 125 and the bytes 74.
#include "moe_internal.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kRows = 64;          // rows of a tile
constexpr int kShrinkK = 64;       // K elements of a shrink stage
constexpr int kStages = 4;         // stages of the shrink's ring
constexpr int kGradStages = 3;     // of the grad's: room for three CTAs on an SM up to rank 64
constexpr int kGradCols = 128;     // columns of a grad CTA
constexpr int kGradRows = 32;      // tokens of a grad stage
constexpr int kGradFlush = 4;      // grad stages between additions to the sums
constexpr int kMaxSlices = 8;      // K slices of a shrink (CTAs of a cluster)

// bf16 parts of an operand: of type T itself, and of an fp32 one
template <typename T>
struct Parts;
template <>
struct Parts<__nv_bfloat16> {
    static constexpr int self = 1, f32 = 3;
};
template <>
struct Parts<float> {
    static constexpr int self = 3, f32 = 3;
};
template <typename TA, typename T>
constexpr int act_parts() {
    return std::is_same<TA, T>::value ? Parts<T>::self : Parts<T>::f32;
}

struct Tile {
    int32_t adapter, pos, rows, pad;  // adapter n_adapters: the tokens that have none
};

struct Plan {
    int32_t* perm;      // [N] token at each sorted position
    int32_t* seg;       // [n_adapters + 2] first position of each adapter; tokens without one last
    Tile* tiles;        // tiles of at most kRows rows, one adapter each
    int32_t* n_tiles;
    int32_t* one_group; // {0, N}, {0, ceil(N / 128)}, {0, ceil(N / 256)}: all rows as one group of the GEMMs
    unsigned long long* counters;
};

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"((uint32_t)__cvta_generic_to_shared(p)));
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// v = sum of P bf16 parts, each the rounding of what the ones before leave.  The
// first of three is the value cut off, so that the largest finite ones stay
// finite (rounded, they would be infinite); the parts are exact all the same.
// The first of two is rounded, which keeps 16 bits where cutting off keeps 15,
// and cut off only where it would be infinite.
// A value that is not finite is its first part; the others are 0.
template <int P>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&out)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        out[i] = P == 3 && i == 0 ? __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632) : pack2(a, b);
        if (i + 1 < P) {
            float left_a = a - __uint_as_float(out[i] << 16), left_b = b - __uint_as_float(out[i] & 0xffff0000u);
            const float both = left_a + left_b;
            if (i == 0 && !isfinite(both)) {  // one was not finite, or rounded to an infinity (rare)
                if (P != 3) {
                    const uint32_t cut_a = __float_as_uint(a) & 0xffff0000u, cut_b = __float_as_uint(b) & 0xffff0000u;
                    if (isfinite(a) && !isfinite(left_a)) {
                        out[i] = (out[i] & 0xffff0000u) | cut_a >> 16;
                        left_a = a - __uint_as_float(cut_a);
                    }
                    if (isfinite(b) && !isfinite(left_b)) {
                        out[i] = (out[i] & 0xffffu) | cut_b;
                        left_b = b - __uint_as_float(cut_b);
                    }
                }
                // cut off, a NaN might pass for an infinity
                if (a != a) out[i] |= 0x7fc0u;
                if (b != b) out[i] |= 0x7fc00000u;
                a = isfinite(left_a) ? left_a : 0.f;
                b = isfinite(left_b) ? left_b : 0.f;
            } else {
                a = left_a;
                b = left_b;
            }
        }
    }
}

// eight consecutive elements as P parts of four packed pairs
template <int P>
__device__ __forceinline__ void load8_parts(const __nv_bfloat16* p, bool in, uint4 (&out)[P]) {
    static_assert(P == 1, "16-bit operands are one part");
    out[0] = in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
}
template <int P>
__device__ __forceinline__ void split8(float4 lo, float4 hi, uint4 (&out)[P]) {
    uint32_t a[P], b[P], c[P], d[P];
    split2<P>(lo.x, lo.y, a);
    split2<P>(lo.z, lo.w, b);
    split2<P>(hi.x, hi.y, c);
    split2<P>(hi.z, hi.w, d);
#pragma unroll
    for (int i = 0; i < P; ++i) out[i] = make_uint4(a[i], b[i], c[i], d[i]);
}
template <int P>
__device__ __forceinline__ void load8_parts(const float* p, bool in, uint4 (&out)[P]) {
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    split8<P>(in ? *reinterpret_cast<const float4*>(p) : zero, in ? *reinterpret_cast<const float4*>(p + 4) : zero, out);
}

// 16 bytes global -> shared, asynchronously; zeros where !in
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Every kernel here begins with it: the next one of the call may get ready, and
// what the ones before have written is there from here on.
__device__ __forceinline__ void in_turn() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// whether the product of parts i and j counts beside operands of PA and PB parts
template <int PA, int PB>
__device__ __forceinline__ constexpr bool counts(int i, int j) {
    return i + j < (PA > PB ? PA : PB);
}

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of the tokens by adapter, by one CTA.  Warp w
// walks tokens [w chunk, (w+1) chunk) in order; lanes with the same adapter
// take consecutive places.  Ids out of range count as none and are reported.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) adapter_plan_kernel(const int32_t* ids, int N, int n_adapters, Plan p) {
    extern __shared__ int32_t sm[];
    in_turn();
    const int nb = n_adapters + 1;
    int32_t* cnt = sm;               // [32][nb] tokens of bucket b before warp w's next one
    int32_t* first = sm + 32 * nb;   // [nb + 1]
    int32_t* tile0 = first + nb + 1; // [nb + 1]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < 32 * nb; i += 1024) cnt[i] = 0;
    if (tid < CNT_COUNT) p.counters[tid] = 0ull;
    __syncthreads();
    const int chunk = ((N + 31) / 32 + 31) / 32 * 32;
    const int t0 = warp * chunk, t1 = min(N, t0 + chunk);
    bool bad = false;
    // buckets of 8 x 32 tokens from b on, loaded together
    auto buckets = [&](int b, int (&id)[8]) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int t = b + q * 32 + lane;
            id[q] = t < t1 ? ids[t] : -2;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const bool in = b + q * 32 + lane < t1;
            if (in && (id[q] < -1 || id[q] >= n_adapters)) bad = true;
            id[q] = !in ? -1 : (id[q] < 0 || id[q] >= n_adapters ? n_adapters : id[q]);
        }
    };
    for (int b = t0; b < t1; b += 256) {
        int id[8];
        buckets(b, id);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (b + q * 32 >= t1) break;
            const unsigned same = __match_any_sync(0xffffffffu, id[q]);
            if (id[q] >= 0 && lane == __ffs(same) - 1) cnt[warp * nb + id[q]] += __popc(same);
            __syncwarp();
        }
    }
    if (bad) atomicOr(p.counters + CNT_DEVICE_ERROR, (unsigned long long)DEVERR_BOUNDS);
    __syncthreads();
    for (int b = warp; b < nb; b += 32) {  // exclusive over the warps (a lane each), total in first[b]
        const int c = cnt[lane * nb + b];
        int v = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        cnt[lane * nb + b] = v - c;
        if (lane == 31) first[b] = v;
    }
    __syncthreads();
    if (warp == 0) {
        int rows = 0, tiles = 0;
        for (int b = 0; b < nb; b += 32) {
            const int c = b + lane < nb ? first[b + lane] : 0, t = (c + kRows - 1) / kRows;
            int sc = c, st = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, sc, o), v = __shfl_up_sync(0xffffffffu, st, o);
                if (lane >= o) {
                    sc += u;
                    st += v;
                }
            }
            __syncwarp();
            if (b + lane < nb) {
                first[b + lane] = rows + sc - c;
                tile0[b + lane] = tiles + st - t;
            }
            rows += __shfl_sync(0xffffffffu, sc, 31);
            tiles += __shfl_sync(0xffffffffu, st, 31);
        }
        if (lane == 0) {
            first[nb] = rows;
            tile0[nb] = tiles;
            *p.n_tiles = tiles;
            p.one_group[0] = 0;
            p.one_group[1] = N;
            p.one_group[2] = 0;
            p.one_group[3] = (N + 127) / 128;
            p.one_group[4] = 0;
            p.one_group[5] = (N + 255) / 256;
        }
    }
    __syncthreads();
    for (int b = tid; b <= nb; b += 1024) p.seg[b] = first[b];
    for (int i = tid; i < tile0[nb]; i += 1024) {
        int lo = 0, hi = nb - 1;  // the last bucket whose tiles begin at or before i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tile0[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        const int pos = first[lo] + (i - tile0[lo]) * kRows;
        p.tiles[i] = {lo, pos, min(kRows, first[lo + 1] - pos), 0};
    }
    for (int b = t0; b < t1; b += 256) {
        int id[8];
        buckets(b, id);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (b + q * 32 >= t1) break;
            const unsigned same = __match_any_sync(0xffffffffu, id[q]);
            int at = 0;
            if (id[q] >= 0) at = first[id[q]] + cnt[warp * nb + id[q]] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (id[q] >= 0) {
                if (lane == __ffs(same) - 1) cnt[warp * nb + id[q]] += __popc(same);
                p.perm[at] = b + q * 32 + lane;
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------------------
// shrink: out[pos, q] = s_a sum_k X[tok(pos), k] M_a(q, k) as parts.
//   NN = false: M_a is A_a [r, K] (x -> u);  NN = true: M_a is B_a [K, r] (dy -> v)
// A CTA has one tile and one of the cluster's K slices.  Stages of 64 K come
// through a ring of asynchronous copies (the rows are gathered there); each of
// the 8 warps has 16 rows and one of a stage's two steps of 32 K.  (Four warps
// of 32 rows read the adapter half as often from shared memory, but left two
// warps a scheduler to hide everything behind.)  A lane reads 8 consecutive K
// elements of a row and feeds them to two MMAs, the adapter's elements in the
// same order of K.  The cluster's CTAs add their sums in slice order through
// distributed shared memory.
// Measured: u of 4096 x 4096 bf16, r = 16, 14 to 19 us (33.5 MB); u and v of 8192 x
// 4096, r = 64, 97 us (201 MB): the MMAs that meet a stage, 2 CTAs of 8 warps on an
// SM, take longer than its bytes.
// ---------------------------------------------------------------------------
struct ShrinkArgs {
    const void* X;
    const void* M;
    const float* scale;
    int K, r, n_adapters, slice;
    int64_t N;
    __nv_bfloat16* out;  // [parts][N][r]
    Plan p;
};

// row pitches that keep the lanes' reads apart: 16-bit rows of 64 elements, 64
// bytes above a multiple of 128 (a quarter-warp reads 2 rows x 64 bytes);
// 32-bit ones, 16 above (2 rows x 4 x 16 bytes, 32 apart); an adapter's rows of
// r ranks, 16 above
template <typename TA>
constexpr int shrink_x_pitch() { return sizeof(TA) == 2 ? kShrinkK * 2 + 64 : kShrinkK * 4 + 16; }
template <typename T, bool NN>
__host__ __device__ constexpr int shrink_m_pitch(int r) {
    return NN ? r * (int)sizeof(T) + 16 : shrink_x_pitch<T>();
}
template <typename T, typename TA, bool NN>
__host__ __device__ constexpr int shrink_stage(int r) {
    return kRows * shrink_x_pitch<TA>() + (NN ? kShrinkK : r) * shrink_m_pitch<T, NN>(r);
}

constexpr int kShrinkThreads = 256;
constexpr int kShrinkFlush = 4;    // stages between additions to the sums

template <typename T, typename TA, bool NN, int NQ>
__device__ __forceinline__ void shrink(const ShrinkArgs& a) {
    constexpr int PA = act_parts<TA, T>(), PB = Parts<T>::self, PF = Parts<T>::f32;
    constexpr int kXPitch = shrink_x_pitch<TA>();
    extern __shared__ __align__(128) uint8_t smem[];
    const cg::cluster_group cluster = cg::this_cluster();
    if ((int)blockIdx.x >= *a.p.n_tiles) return;  // the same for the whole cluster
    const Tile tile = a.p.tiles[blockIdx.x];
    if (tile.adapter >= a.n_adapters) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int r = a.r, m_pitch = shrink_m_pitch<T, NN>(r), stage_bytes = shrink_stage<T, TA, NN>(r);
    const int k_beg = blockIdx.y * a.slice, k_end = min(a.K, k_beg + a.slice);
    const int chunks = k_beg < k_end ? (k_end - k_beg + kShrinkK - 1) / kShrinkK : 0;
    // this thread's copies of a stage, each with a source that moves on by a
    // stage.  X: 16-byte piece xp of rows xr, xr + XS, ... (zeros past the tile)
    constexpr int XPIECES = kShrinkK * (int)sizeof(TA) / 16, XS = kShrinkThreads / XPIECES, XN = kRows / XS;
    const int xp = tid % XPIECES, xr = tid / XPIECES, xk = xp * (16 / (int)sizeof(TA));
    const TA* xsrc[XN];
    bool xhave[XN];
#pragma unroll
    for (int i = 0; i < XN; ++i) {
        const int q = xr + i * XS;
        xhave[i] = q < tile.rows;
        xsrc[i] = static_cast<const TA*>(a.X) + (xhave[i] ? (int64_t)a.p.perm[tile.pos + q] * a.K : 0) + k_beg + xk;
    }
    // M: pieces tid, tid + 256, ... of the [r][64] (NN: [64][r]) block
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int MN = (NQ * 8 * kShrinkK / E + kShrinkThreads - 1) / kShrinkThreads;
    const T* const M = static_cast<const T*>(a.M) + (int64_t)tile.adapter * r * a.K + (int64_t)k_beg * (NN ? r : 1);
    const T* msrc[MN];
    int mdst[MN], mk[MN];  // byte offset in the stage; first K of the piece (no such piece: past all)
#pragma unroll
    for (int i = 0; i < MN; ++i) {
        const int per = NN ? r / E : kShrinkK / E, at = tid + i * kShrinkThreads, major = at / per, minor = at % per * E;
        const bool have = major < (NN ? kShrinkK : r);
        mk[i] = have ? (NN ? major : minor) : 1 << 30;
        msrc[i] = M + (have ? (NN ? (int64_t)major * r : (int64_t)major * a.K) + minor : 0);
        // NN: K rows in the order that puts the four lanes' rows next to one another
        const int row = NN ? (major & 32) + (major & 7) * 4 + (major >> 3 & 3) : major;
        mdst[i] = kRows * kXPitch + row * m_pitch + minor * (int)sizeof(T);
    }
    const uint32_t ring = smem_addr(smem), xdst = xr * kXPitch + xp * 16;
    uint32_t to = ring;
    int left = k_end - k_beg;  // K from the next stage to fill on
    auto fill = [&]() {
        if (left > 0) {
            const bool whole = left >= kShrinkK;
#pragma unroll
            for (int i = 0; i < XN; ++i) {
                const bool in = xhave[i] && (whole || xk < left);
                copy16(to + xdst + i * XS * kXPitch, whole || in ? xsrc[i] : a.X, in);
                xsrc[i] += kShrinkK;
            }
#pragma unroll
            for (int i = 0; i < MN; ++i) {
                const bool in = whole || mk[i] < left;
                if (mk[i] < kShrinkK) copy16(to + mdst[i], in ? msrc[i] : M, in);
                msrc[i] += NN ? kShrinkK * r : kShrinkK;
            }
            left -= kShrinkK;
            to = to + stage_bytes == ring + kStages * stage_bytes ? ring : to + stage_bytes;
        }
        copies_commit();
    };
#pragma unroll
    for (int c = 0; c < kStages - 1; ++c) fill();
    const int row0 = (warp & 3) * 16, step = warp >> 2;
    float sum[NQ][4] = {}, acc[NQ][4] = {};
    auto flush = [&]() {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sum[n][e] += acc[n][e];
                acc[n][e] = 0.f;
            }
    };
    for (int c = 0; c < chunks; ++c) {
        copies_wait<kStages - 2>();
        __syncthreads();
        fill();
        const uint8_t* xs = smem + c % kStages * stage_bytes;
        const uint8_t* ms = xs + kRows * kXPitch;
        if (row0 < tile.rows) {  // else none of this warp's rows is in the tile
            uint4 x[2][PA];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                load8_parts<PA>(reinterpret_cast<const TA*>(xs + (row0 + g + 8 * i) * kXPitch) + step * 32 + t * 8, true, x[i]);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                if (n * 8 >= r) break;
                uint4 b[PB];
                if constexpr (!NN) {
                    load8_parts<PB>(reinterpret_cast<const T*>(ms + (n * 8 + g) * m_pitch) + step * 32 + t * 8, true, b);
                } else if constexpr (sizeof(T) == 2) {
                    const int m = lane >> 3, i = lane & 7;
                    uint32_t v[4];
                    ldmatrix_x4_trans(v, ms + (step * 32 + ((i & 1) + 2 * m) * 4 + (i >> 1)) * m_pitch + n * 16);
                    b[0] = make_uint4(v[0], v[1], v[2], v[3]);
                } else {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = *reinterpret_cast<const float*>(ms + (step * 32 + e * 4 + t) * m_pitch + (n * 8 + g) * 4);
                    split8<PB>(make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7]), b);
                }
                // small products first
#pragma unroll
                for (int level = (PA > PB ? PA : PB) - 1; level >= 0; --level)
#pragma unroll
                    for (int j = 0; j < PB; ++j) {
                        const int i = level - j;
                        if (i < 0 || i >= PA) continue;
                        const uint4 &lo = x[0][i], &hi = x[1][i];
                        mma_bf16(acc[n], lo.x, hi.x, lo.y, hi.y, b[j].x, b[j].y);
                        mma_bf16(acc[n], lo.z, hi.z, lo.w, hi.w, b[j].z, b[j].w);
                    }
            }
        }
        if (c % kShrinkFlush == kShrinkFlush - 1) flush();
    }
    flush();
    // the cluster's sums, slice by slice (and step by step), then the parts
    copies_wait<0>();
    __syncthreads();
    float* mine = reinterpret_cast<float*>(smem);  // [2 steps][64][r]
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        if (n * 8 >= r) break;
        const int at = (step * kRows + row0 + g) * r + n * 8 + 2 * t;
        *reinterpret_cast<float2*>(mine + at) = make_float2(sum[n][0], sum[n][1]);
        *reinterpret_cast<float2*>(mine + at + 8 * r) = make_float2(sum[n][2], sum[n][3]);
    }
    cluster.sync();
    const int slices = cluster.num_blocks(), rank = cluster.block_rank();
    const float scale = a.scale[tile.adapter];
    const int pairs = tile.rows * r / 2;
    for (int i = rank * kShrinkThreads + tid; i < pairs; i += kShrinkThreads * slices) {
        float2 s = make_float2(0.f, 0.f);
        for (int q = 0; q < slices; ++q) {
            const float* theirs = cluster.map_shared_rank(mine, q) + 2 * i;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float2 v = *reinterpret_cast<const float2*>(theirs + m * kRows * r);
                s.x += v.x;
                s.y += v.y;
            }
        }
        uint32_t out[PF];
        split2<PF>(s.x * scale, s.y * scale, out);
#pragma unroll
        for (int j = 0; j < PF; ++j)
            *reinterpret_cast<uint32_t*>(a.out + ((int64_t)j * a.N + tile.pos) * r + 2 * i) = out[j];
    }
    cluster.sync();  // the others have read this CTA's sums
}

template <typename T, int NQ>
__global__ void __launch_bounds__(kShrinkThreads) adapter_shrink_kernel(const __grid_constant__ ShrinkArgs u) {
    in_turn();
    shrink<T, T, false, NQ>(u);
}
// u and v in one launch: neither needs the other.  v, the longer one, goes first,
// and u's CTAs fill in behind it
template <typename T, int NQ>
__global__ void __launch_bounds__(kShrinkThreads)
    adapter_shrink_both_kernel(const __grid_constant__ ShrinkArgs u, const __grid_constant__ ShrinkArgs v) {
    in_turn();
    if (blockIdx.z == 0) shrink<T, float, true, NQ>(v);
    else shrink<T, T, false, NQ>(u);
}

// ---------------------------------------------------------------------------
// expand: out[tok(pos), j] = base[tok, j] (+ out[tok, j]) + sum_q in[pos, q] M_a(q, j)
//   NN = false: M_a is B_a [J, r] (u -> y);  NN = true: M_a is A_a [r, J] (v -> dx)
// A CTA has one tile and a span of columns; each warp 16 of the rows, their
// parts of u in registers throughout, the span's part of the adapter in shared
// memory.  Of 32 columns a lane has 4 t .. 4 t + 3 and the same 16 further on, of
// two rows (the four MMA tiles take the columns in that order), so a row is read
// and written in 64 consecutive bytes; what is added to is fetched two steps
// ahead.
// Measured: 4096 x 4096, r = 16, read and written in 26 us (134 MB, 5.2 TB/s).
// ---------------------------------------------------------------------------
struct ExpandArgs {
    const __nv_bfloat16* in;  // [parts][N][r]
    const void* M;
    const float* base;        // nullable; may be out (what a projection left there counts as base)
    const float* base2;       // nullable: added too
    float* out;
    int J, r, n_adapters, span;
    int64_t N;
    Plan p;
};

// bytes between rows of r elements so that a half-warp's 8-byte reads (4 rows x
// 32 bytes) do not collide: 32 above a multiple of 64
__host__ __device__ constexpr int expand_pitch(int r) { return (2 * r + 31) / 64 * 64 + 32; }

// shared memory of a span of columns of an adapter
template <typename T, bool NN, int NK>
__host__ __device__ constexpr int expand_part(int span) {
    return NN ? NK * 16 * (span * 2 + 16) : span * expand_pitch(NK * 16);
}

// as many CTAs on an SM as the parts of u leave registers for
template <typename T, bool NN, int NK>
__global__ void __launch_bounds__(128, NK == 1 ? 4 : NK <= 4 ? 3 : 2) adapter_expand_kernel(const __grid_constant__ ExpandArgs a) {
    constexpr int PB = Parts<T>::self, PF = Parts<T>::f32;
    constexpr int R = NK * 16;
    const int pitch = NN ? a.span * 2 + 16 : expand_pitch(R), part_bytes = expand_part<T, NN, NK>(a.span);
    extern __shared__ __align__(128) uint8_t smem[];
    in_turn();
    if ((int)blockIdx.x >= *a.p.n_tiles) return;
    const Tile tile = a.p.tiles[blockIdx.x];
    const bool none = tile.adapter >= a.n_adapters;
    // tokens without an adapter: base alone
    if (none && a.base == a.out && !a.base2) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int r = a.r, J = a.J;
    const T* M = static_cast<const T*>(a.M) + (none ? 0 : (int64_t)tile.adapter * r * J);
    const int jb = blockIdx.y * a.span, cols = min(a.span, J - jb);
    // place of column j among the span's: tiles 0 and 1 (of 16 columns on: 2 and 3) take pairs in turn
    auto place = [](int j) { return (j & ~15) + (j >> 1 & 1) * 8 + (j >> 2 & 3) * 2 + (j & 1); };
    if (!none) {
        // 128 columns at a time, this thread's 2 NK pieces of 8 elements together
#pragma unroll 1
        for (int c = 0; c < cols; c += 128) {
            uint4 v[2 * NK][PB];
            if (NN) {
                const int j = c + tid % 16 * 8, k0 = tid / 16;
#pragma unroll
                for (int i = 0; i < 2 * NK; ++i) {
                    const int k = k0 + 8 * i;
                    load8_parts<PB>(M + (int64_t)k * J + jb + j, k < r && j < cols, v[i]);
                }
#pragma unroll
                for (int i = 0; i < 2 * NK; ++i) {
                    // K rows in the order that puts the four lanes' rows next to one another
                    const int k = k0 + 8 * i;
                    uint8_t* at = smem + ((k & ~15) + (k & 3) * 4 + (k >> 2 & 3)) * pitch + place(j) * 2;
#pragma unroll
                    for (int q = 0; q < PB; ++q) {
                        *reinterpret_cast<uint2*>(at + q * part_bytes) = make_uint2(v[i][q].x, v[i][q].z);
                        *reinterpret_cast<uint2*>(at + q * part_bytes + 16) = make_uint2(v[i][q].y, v[i][q].w);
                    }
                }
            } else {
                const int k = tid % (2 * NK) * 8, j0 = c + tid / (2 * NK);
#pragma unroll
                for (int i = 0; i < 2 * NK; ++i) {
                    const int j = j0 + i * (64 / NK);
                    load8_parts<PB>(M + (int64_t)(jb + j) * r + k, k < r && j < cols, v[i]);
                }
#pragma unroll
                for (int i = 0; i < 2 * NK; ++i)
#pragma unroll
                    for (int q = 0; q < PB; ++q)
                        *reinterpret_cast<uint4*>(smem + q * part_bytes + place(j0 + i * (64 / NK)) * pitch + k * 2) = v[i][q];
            }
        }
    }
    // rows g and g + 8 of the warp; one past the tile reads the tile's first and writes nothing
    const float* base[2];
    int64_t at[2];
    bool have[2];
    uint32_t u[PF][NK][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int q = warp * 16 + g + 8 * i;
        have[i] = q < tile.rows;
        at[i] = (int64_t)a.p.perm[tile.pos + (have[i] ? q : 0)] * J + jb + 4 * t;
        base[i] = a.base + at[i];
#pragma unroll
        for (int j = 0; j < PF; ++j)
#pragma unroll
            for (int s = 0; s < NK; ++s) {
                // K in the order (4 t .. 4 t + 3): 8 bytes of a row
                const int k = s * 16 + 4 * t;
                uint2 v = make_uint2(0, 0);
                if (have[i] && k < r && !none)
                    v = *reinterpret_cast<const uint2*>(a.in + ((int64_t)j * a.N + tile.pos + q) * r + k);
                u[j][s][i] = v.x;
                u[j][s][2 + i] = v.y;
            }
    }
    const int lim = cols - 4 * t;
    const bool based = a.base != nullptr;
    // what 32 columns from n0 on are added to: 4 and 4 of two rows
    auto fetch = [&](int n0, float4 (&v)[2][2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[i][h] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (based && n0 + 16 * h < lim) v[i][h] = *reinterpret_cast<const float4*>(base[i] + n0 + 16 * h);
            }
    };
    float4 next[2][2][2];  // the next two steps'
    fetch(0, next[0]);
    fetch(32, next[1]);
    __syncthreads();
    if (warp * 16 >= tile.rows) return;  // none of this warp's rows is in the tile
#pragma unroll 2
    for (int n0 = 0; n0 < cols; n0 += 32) {
        float4 add[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                add[i][h] = next[0][i][h];
                next[0][i][h] = next[1][i][h];
            }
        fetch(n0 + 64, next[1]);
        float acc[4][4] = {};
        if (!none) {
#pragma unroll
            for (int s = 0; s < NK; ++s) {
                uint32_t b[PB][4][2];
#pragma unroll
                for (int q = 0; q < PB; ++q) {
                    if (NN) {
                        // two column tiles at a time: (b0, b1) of each
                        const int m = lane >> 3, i = lane & 7;
                        const uint8_t* p = smem + q * part_bytes +
                                           (s * 16 + ((i & 1) + 2 * (m & 1)) * 4 + (i >> 1)) * pitch +
                                           (n0 + (m >> 1) * 8) * 2;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[4];
                            ldmatrix_x4_trans(v, p + h * 32);
                            b[q][2 * h][0] = v[0];
                            b[q][2 * h][1] = v[1];
                            b[q][2 * h + 1][0] = v[2];
                            b[q][2 * h + 1][1] = v[3];
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const uint2 v = *reinterpret_cast<const uint2*>(
                                smem + q * part_bytes + (n0 + n * 8 + g) * pitch + (s * 16 + 4 * t) * 2);
                            b[q][n][0] = v.x;
                            b[q][n][1] = v.y;
                        }
                    }
                }
#pragma unroll
                for (int level = (PF > PB ? PF : PB) - 1; level >= 0; --level)  // small products first
#pragma unroll
                    for (int q = 0; q < PB; ++q) {
                        const int j = level - q;
                        if (j < 0 || j >= PF) continue;
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            mma_bf16(acc[n], u[j][s][0], u[j][s][1], u[j][s][2], u[j][s][3], b[q][n][0], b[q][n][1]);
                    }
            }
        }
        // tiles 2 h and 2 h + 1 have the pairs of this lane's four columns at 16 h
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!have[i] || n0 + 16 * h >= lim) continue;
                float4 v = make_float4(add[i][h].x + acc[2 * h][2 * i], add[i][h].y + acc[2 * h][2 * i + 1],
                                       add[i][h].z + acc[2 * h + 1][2 * i], add[i][h].w + acc[2 * h + 1][2 * i + 1]);
                if (a.base2) {
                    const float4 w = *reinterpret_cast<const float4*>(a.base2 + at[i] + n0 + 16 * h);
                    v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
                }
                *reinterpret_cast<float4*>(a.out + at[i] + n0 + 16 * h) = v;
            }
    }
}

// ---------------------------------------------------------------------------
// grad: G_a(q, j) = sum over adapter a's tokens of in[pos, q] Z[tok(pos), j]
//   TRANS = false: dA_a [r, J] from v and x;  TRANS = true: dB_a [J, r] from u and dy
// A CTA has 128 columns and a range of the sorted tokens that have an adapter (see
// ranges_of), the same for every CTA of the row whatever the adapters' shares (cut by adapter instead, the largest
// one's CTAs ran alone at the end: 143 against 77 us for dB of 8192 tokens of
// four uneven adapters, r = 64, d = 4096).  An adapter that lies in one range is
// written to its place; one that continues in others leaves a partial sum in each,
// which the reduction adds in order.  Only the first and the last adapter of a
// range can, so it has a place for one that began before it and a place for one
// that begins in it and goes on.  Each
// warp has 32 of the columns and all ranks.  The tokens' parts of u or v, which
// all warps need, and their places come through a ring of asynchronous copies;
// a row of Z is used by one warp only and goes from global memory to its
// registers a stage ahead: a lane reads 4 consecutive columns of four rows, and
// the four MMA tiles take the columns in that order, so a lane's results are 8
// consecutive columns too.
// Measured: both gradients of 8192 tokens, r = 64, d = 4096, 162 us with the tensor
// pipe busy 45% of the time: six of nine products of parts for dB, three for dA, at
// 12 warps an SM (the sums of a thread take 64 registers and the fetched rows 32).
// ---------------------------------------------------------------------------
struct GradArgs {
    const __nv_bfloat16* in;  // [parts][N][r]
    const void* Z;
    float* out;               // [n_adapters][r J]
    float* part;              // [ranges][2][r J]: partial sums of the adapter that began before the range
                              // and of the one that begins in it and goes on
    int J, r, n_adapters;
    int ranges;
    int64_t N;
    Plan p;
};

template <int PF, int MT>
constexpr int grad_stage() { return PF * kGradRows * (MT * 32 + 16) + kGradRows * 4; }
template <int PF, int MT>
constexpr size_t grad_smem() { return (size_t)kGradStages * grad_stage<PF, MT>() + (size_t)MT * 16 * 128 * 4; }

// 4 consecutive elements as they are in memory
template <typename TZ>
struct Raw4;
template <>
struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void zero() { v = make_uint2(0, 0); }
};
// column n of two rows as P packed parts
template <int P>
__device__ __forceinline__ void pair_parts(const Raw4<float>& a, const Raw4<float>& b, int n, uint32_t (&out)[P]) {
    split2<P>(n == 0 ? a.v.x : n == 1 ? a.v.y : n == 2 ? a.v.z : a.v.w,
              n == 0 ? b.v.x : n == 1 ? b.v.y : n == 2 ? b.v.z : b.v.w, out);
}
template <int P>
__device__ __forceinline__ void pair_parts(const Raw4<__nv_bfloat16>& a, const Raw4<__nv_bfloat16>& b, int n,
                                           uint32_t (&out)[P]) {
    static_assert(P == 1, "16-bit operands are one part");
    out[0] = __byte_perm(n < 2 ? a.v.x : a.v.y, n < 2 ? b.v.x : b.v.y, n & 1 ? 0x7632 : 0x5410);
}

// The ranges that `tokens` adapted tokens go in: as many as the host launched CTAs
// for, which knows only how many tokens there are in all, but none without a
// token.  An empty range would write nothing, and the reduction reads all ranges
// from an adapter's first token to its last
__device__ __forceinline__ int ranges_of(const GradArgs& a, int tokens) { return min(a.ranges, tokens); }

template <typename T, typename TZ, bool TRANS, int MT>
__device__ __forceinline__ void grad(const GradArgs& a, int col_block, int range) {
    constexpr int PZ = act_parts<TZ, T>(), PF = Parts<T>::f32;
    constexpr int kInPitch = MT * 32 + 16, kInPart = kGradRows * kInPitch, kStage = grad_stage<PF, MT>();
    constexpr int STEPS = kGradRows / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    float* sums = reinterpret_cast<float*>(smem + kGradStages * kStage);  // [MT * 16][128 threads]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int r = a.r, J = a.J;
    const int tokens = a.p.seg[a.n_adapters];  // those that have an adapter
    const int ranges = ranges_of(a, tokens);
    if (range >= ranges) return;
    const int lo = (int)((int64_t)tokens * range / ranges), hi = (int)((int64_t)tokens * (range + 1) / ranges);
    const int col = col_block * kGradCols + warp * 32 + 4 * g;  // this lane's columns of Z
    const TZ* Z = static_cast<const TZ*>(a.Z) + col;
    const bool col_in = col < J;
    // the adapter of position lo: the last one that begins at or before it
    int adapter = 0;
    for (int top = a.n_adapters - 1; adapter < top;) {
        const int mid = (adapter + top + 1) >> 1;
        if (a.p.seg[mid] <= lo) adapter = mid;
        else top = mid - 1;
    }
    // this thread's pieces of a stage: 8 ranks of rows ir, ir + IS, ...
    constexpr int IP = MT * 2, IS = 128 / IP, IN = (kGradRows + IS - 1) / IS;
    const int iq = tid % IP * 8, ir = tid / IP;
    for (int beg = lo; beg < hi; ++adapter) {
        const int seg0 = a.p.seg[adapter], seg_end = a.p.seg[adapter + 1];
        if (seg_end <= beg) continue;  // an adapter without tokens
        const int seg1 = min(seg_end, hi), c1 = (seg1 - beg + kGradRows - 1) / kGradRows;
        auto fill = [&](int c) {
            if (c < c1) {
                const uint32_t st = smem_addr(smem) + c % kGradStages * kStage;
                const int pos = beg + c * kGradRows;
#pragma unroll
                for (int i = 0; i < IN; ++i) {
                    const int row = ir + i * IS;
                    if (row >= kGradRows) break;
                    const bool in = pos + row < seg1 && iq < r;
#pragma unroll
                    for (int j = 0; j < PF; ++j)
                        copy16(st + j * kInPart + row * kInPitch + iq * 2,
                               in ? a.in + ((int64_t)j * a.N + pos + row) * r + iq : a.in, in);
                }
                if (tid < kGradRows)  // 4 bytes each: the places need not be 16-byte aligned
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(st + PF * kInPart + tid * 4),
                                 "l"(a.p.perm + (pos + tid < seg1 ? pos + tid : 0)), "r"(pos + tid < seg1 ? 4 : 0)
                                 : "memory");
            }
            copies_commit();
        };
        // rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of each step of 16 tokens
        auto fetch = [&](int c, Raw4<TZ> (&z)[STEPS][4]) {
            const int32_t* tok = reinterpret_cast<const int32_t*>(smem + c % kGradStages * kStage + PF * kInPart);
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = s * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
                    if (col_in && beg + c * kGradRows + row < seg1) z[s][i].load(Z + (int64_t)tok[row] * J);
                    else z[s][i].zero();
                }
        };
#pragma unroll
        for (int c = 0; c < kGradStages - 1; ++c) fill(c);
        float acc[MT][4][4] = {};
        auto flush = [&](bool first, bool last) {
#pragma unroll
            for (int i = 0; i < MT * 16; ++i) {
                float& v = acc[i / 16][i / 4 % 4][i % 4];
                if (!first) v += sums[i * 128 + tid];
                if (!last) {
                    sums[i * 128 + tid] = v;
                    v = 0.f;
                }
            }
        };
        Raw4<TZ> z[STEPS][4];
        copies_wait<kGradStages - 2>();
        __syncthreads();
        fetch(0, z);
        bool first = true;
        for (int c = 0; c < c1; ++c) {
            copies_wait<kGradStages - 3>();  // this stage and the next
            __syncthreads();
            fill(c + kGradStages - 1);
            Raw4<TZ> ahead[STEPS][4];
            if (c + 1 < c1) fetch(c + 1, ahead);
            const uint8_t* st = smem + c % kGradStages * kStage;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int m = lane >> 3, i = lane & 7;
                uint32_t b[4][2][PZ];
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) pair_parts<PZ>(z[s][2 * h], z[s][2 * h + 1], n, b[n][h]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int j = PF - 1; j >= 0; --j) {
                        // A: (m 0-7, k 0-7), (m 8-15, k 0-7), (m 0-7, k 8-15), (m 8-15, k 8-15)
                        uint32_t v[4];
                        ldmatrix_x4_trans(v, st + j * kInPart + (s * 16 + (m >> 1) * 8 + i) * kInPitch +
                                                 (mt * 16 + (m & 1) * 8) * 2);
#pragma unroll
                        for (int q = PZ - 1; q >= 0; --q) {
                            if (!counts<PF, PZ>(j, q)) continue;
#pragma unroll
                            for (int n = 0; n < 4; ++n)
                                mma_bf16(acc[mt][n], v[0], v[1], v[2], v[3], b[n][0][q], b[n][1][q]);
                        }
                    }
                }
            }
            if (c % kGradFlush == kGradFlush - 1 && c + 1 < c1) {
                flush(first, false);
                first = false;
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) z[s][i] = ahead[s][i];
        }
        flush(first, true);
        copies_wait<0>();
        __syncthreads();  // the ring is the next adapter's
        // tile n has columns 8 t + n and 8 t + 4 + n of the warp's 32
        const bool alone = seg0 >= lo && seg_end <= hi;
        float* out = alone ? a.out + (int64_t)adapter * r * J : a.part + ((int64_t)2 * range + (seg0 >= lo)) * r * J;
        beg = seg1;
        const int j = col_block * kGradCols + warp * 32 + 8 * t;
        if (j < J) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int q = mt * 16 + g + 8 * h;
                    if (q >= r) continue;
                    if (TRANS) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) out[(int64_t)(j + e) * r + q] = acc[mt][e & 3][2 * h + (e >> 2)];
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float4*>(out + (int64_t)q * J + j + 4 * e) =
                                make_float4(acc[mt][0][2 * h + e], acc[mt][1][2 * h + e], acc[mt][2][2 * h + e],
                                            acc[mt][3][2 * h + e]);
                    }
                }
        }
    }
}

// dA and dB in one launch: the first CTAs are dA's
template <typename T, int MT>
__global__ void __launch_bounds__(128, MT <= 4 ? 3 : 2)
    adapter_grad_kernel(const __grid_constant__ GradArgs dA, const __grid_constant__ GradArgs dB) {
    in_turn();
    const int cols_a = (dA.J + kGradCols - 1) / kGradCols, cols_b = (dB.J + kGradCols - 1) / kGradCols;
    const int i = blockIdx.x - cols_a * dA.ranges;
    if (i < 0) grad<T, T, false, MT>(dA, blockIdx.x % cols_a, blockIdx.x / cols_a);
    else grad<T, float, true, MT>(dB, i % cols_b, i / cols_b);
}

// What the ranges left: an adapter's partial sums, range by range, zeros for one
// without tokens.  CTA (i, a, z): some of adapter a's elements of dA or dB.
__global__ void __launch_bounds__(256)
    adapter_reduce_kernel(const __grid_constant__ GradArgs dA, const __grid_constant__ GradArgs dB) {
    in_turn();
    const GradArgs& a = blockIdx.z ? dB : dA;
    const float4* part = reinterpret_cast<const float4*>(a.part);
    float4* out = reinterpret_cast<float4*>(a.out);
    const int64_t n4 = (int64_t)a.r * a.J / 4;
    const int32_t* seg = a.p.seg;
    const int adapter = blockIdx.y, seg0 = seg[adapter], seg1 = seg[adapter + 1];
    const int64_t tokens = seg[a.n_adapters];
    const int ranges = ranges_of(a, (int)tokens);
    float4* to = out + (int64_t)adapter * n4;
    int first = 0, last = -1;
    if (seg0 < seg1) {
        // the ranges of its first and last token; range i ends at tokens (i + 1) / ranges
        auto range_of = [&](int64_t pos) {
            int i = (int)(pos * ranges / tokens);
            while (tokens * (i + 1) / ranges <= pos) ++i;
            return i;
        };
        first = range_of(seg0);
        last = range_of(seg1 - 1);
        if (first == last) return;  // written where it was summed
    }
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = first; q <= last; ++q) {
            const float4 v = part[((int64_t)2 * q + (q == first)) * n4 + i];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        to[i] = s;
    }
}

// dy as two bf16 parts, the operands of W^T dy
__global__ void __launch_bounds__(256) adapter_split_kernel(const float* v, int64_t n, __nv_bfloat16* hi,
                                                            __nv_bfloat16* lo) {
    in_turn();
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 2048) {
        uint4 p[2];
        load8_parts<2>(v + i, true, p);
        *reinterpret_cast<uint4*>(hi + i) = p[0];
        *reinterpret_cast<uint4*>(lo + i) = p[1];
    }
}

// ---------------------------------------------------------------------------
// A few tokens: u's partial sums per token and K slice, then y
// ---------------------------------------------------------------------------
// CTA (slice, token): part[slice][token][q] over the slice's K, warp w the ranks w, w + 4, ...
template <typename T>
__global__ void __launch_bounds__(128)
    adapter_few_shrink_kernel(const T* x, const T* A, const int32_t* ids, int N, int K, int r, int n_adapters, int slice,
                              float* part, unsigned long long* counters) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t = blockIdx.y;
    if (blockIdx.x == 0 && t == 0 && tid < CNT_COUNT) counters[tid] = 0ull;
    const int id = ids[t];
    if (id < 0 || id >= n_adapters) return;
    const int k0 = blockIdx.x * slice, k1 = min(K, k0 + slice);
    const T* M = A + (int64_t)id * r * K;
    float* out = part + ((int64_t)blockIdx.x * N + t) * r;
    for (int q0 = warp; q0 < r; q0 += 16) {  // four ranks at a time
        float acc[4] = {};
        for (int k = k0 + lane * 8; k < k1; k += 256) {
            float xv[8];
            load8(x + (int64_t)t * K + k, xv);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int q = q0 + 4 * i;
                if (q < r) {
                    float m[8];
                    load8(M + (int64_t)q * K + k, m);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[i] = fmaf(xv[e], m[e], acc[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s = acc[i];
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0 && q0 + 4 * i < r) out[q0 + 4 * i] = s;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(128)
    adapter_few_expand_kernel(const float* part, int slices, const T* B, const float* scale, const int32_t* ids, int N,
                              int J, int r, int n_adapters, const float* base, float* out, int add_out,
                              unsigned long long* counters) {
    __shared__ float u[kMaxAdapterRank];
    const int tid = threadIdx.x, t = blockIdx.y, j = blockIdx.x * 128 + tid;
    const int id = ids[t];
    const bool none = id < 0 || id >= n_adapters;
    const int64_t at = (int64_t)t * J + j;
    const float scaled = none ? 0.f : scale[id];
    float s = 0.f;
    if (j < J && base) s = base[at];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (j < J && add_out) s += out[at];
    if (!none) {
        for (int q = tid; q < r; q += 128) {
            float v = 0.f;
            for (int i = 0; i < slices; ++i) v += part[((int64_t)i * N + t) * r + q];
            u[q] = v * scaled;  // the whole sum: parts that cancel may be past the range, scaled
        }
        __syncthreads();
        if (j < J) {
            const T* row = B + ((int64_t)id * J + j) * r;
            float acc = 0.f;
#pragma unroll 4
            for (int q = 0; q < r; q += 8) {
                float m[8];
                load8(row + q, m);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc = fmaf(u[q + e], m[e], acc);
            }
            s += acc;
        }
    } else if (id != -1 && blockIdx.x == 0 && tid == 0) {
        atomicOr(counters + CNT_DEVICE_ERROR, (unsigned long long)DEVERR_BOUNDS);
    }
    if (j < J) out[at] = s;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// an upper bound of the tiles: every adapter (and the tokens without one) may end in a part of a tile
int64_t tile_bound(const moe_adapter_params& p) {
    return p.N / kRows + std::min<int64_t>(p.n_adapters + 1, p.N);
}

// K slices of a shrink of `smem` bytes a CTA: as many CTAs as fit on the GPU at
// once for the likely tiles (up to four on an SM: their registers), at least two
// stages of K each (of the wider operand's K where u and v are made together: cut
// for the narrower, 192 fp32 tokens, 256 and 1184 wide, r = 40, took 78 instead of 36 us)
int shrink_slices(const moe_adapter_params& p, int K, size_t smem) {
    const int64_t tiles = p.N / kRows + (std::min<int64_t>(p.n_adapters, p.N) + 1) / 2;
    const int64_t slots = std::max<int64_t>(1, std::min<int64_t>(p.r <= 16 ? 4 : 2, (227 * 1024) / ((int64_t)smem + 1024))) * num_sms();
    int s = 1;
    while (s * 2 <= kMaxSlices && s * 2 * tiles <= slots && K / (s * 2) >= 2 * kShrinkK) s *= 2;
    return s;
}

// Whether a batch takes the form of one CTA per token.  It reads an adapter once
// for each of its tokens (from L2 mostly), N r (d_in + d_out) elements in all,
// where the sorted tiles cost about 12 to 30 us however few the tokens; measured
// at widths of 1024 and 4096 and ranks of 8 to 64 the two meet at 25 to 50 MB in
// bf16 (32 adapters, d = 4096, r = 16: 64 tokens 7.9 against 17.9 us, 192 tokens
// 19.8 against 18.6) and at 130 MB and more in fp32 (128 tokens 18.5 against 32.0
// us, 256 tokens 32.8 against 33.7).
bool takes_tokens(const moe_adapter_params& p) {
    const int64_t bytes = p.N * p.r * ((int64_t)p.d_in + p.d_out) * (int64_t)esize(p.dtype);
    return p.N <= 32 || (p.N <= 256 && bytes <= (p.dtype == MOE_BF16 ? 32 : 128) * (int64_t)(1 << 20));
}

int few_slices(int64_t N, int K) {
    return (int)std::max<int64_t>(1, std::min<int64_t>({16, 2 * num_sms() / std::max<int64_t>(N, 1), K / 256}));
}

// ranges of tokens of dA and dB: as many as fit on the GPU at once (three CTAs on
// an SM) with the columns' CTAs, of at least 64 tokens or two adapters each where
// every token has an adapter (where fewer have, the kernels' ranges_of).  In
// bf16 a token of dB takes 5/3 of the time of one of dA (both its operands have
// three parts)
void grad_ranges(const moe_adapter_params& p, int& a, int& b) {
    const int64_t slots = 3 * (int64_t)num_sms();
    const int64_t most = std::max<int64_t>({1, p.N / 64, std::min<int64_t>(p.N, p.n_adapters) / 2});
    const int64_t ca = (p.d_in + kGradCols - 1) / kGradCols, cb = (p.d_out + kGradCols - 1) / kGradCols;
    const int wa = 3, wb = p.dtype == MOE_BF16 ? 5 : 3;
    a = (int)std::max<int64_t>(1, std::min(most, slots * wa / (ca * wa + cb * wb)));
    b = (int)std::max<int64_t>(1, std::min(most, (slots - ca * a) / cb));
}

struct Layout {
    size_t counters, perm, seg, tiles, one_group, u, v, hi, lo, part_a, part_b, total;
};

Layout layout_of(const moe_adapter_params& p, bool with_W, bool backward) {
    const size_t N = (size_t)p.N, r = (size_t)p.r;
    const int parts = p.dtype == MOE_BF16 ? Parts<__nv_bfloat16>::f32 : Parts<float>::f32;
    Layout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = up256(off + bytes);
        return o;
    };
    L.counters = take(CNT_COUNT * 8);
    L.perm = take(N * 4);
    L.seg = take(((size_t)p.n_adapters + 2) * 4);
    L.one_group = take(7 * 4);  // and the number of tiles
    L.tiles = take((size_t)tile_bound(p) * sizeof(Tile));
    // u as parts, or (a few tokens) as partial sums
    L.u = take(std::max(N * r * 2 * parts, !backward && takes_tokens(p) ? few_slices(p.N, p.d_in) * N * r * 4 : 0));
    if (backward) {
        L.v = take(N * r * 2 * parts);
        if (with_W && p.dtype == MOE_BF16) {
            L.hi = take(N * (size_t)p.d_out * 2);
            L.lo = take(N * (size_t)p.d_out * 2);
        }
        // two partial sums a range; none in one range
        int ra, rb;
        grad_ranges(p, ra, rb);
        L.part_a = take(ra > 1 ? (size_t)2 * ra * p.d_in * r * 4 : 0);
        L.part_b = take(rb > 1 ? (size_t)2 * rb * p.d_out * r * 4 : 0);
    }
    L.total = off;
    return L;
}

Plan plan_of(const Layout& L, char* ws) {
    Plan p;
    p.counters = reinterpret_cast<unsigned long long*>(ws + L.counters);
    p.perm = reinterpret_cast<int32_t*>(ws + L.perm);
    p.seg = reinterpret_cast<int32_t*>(ws + L.seg);
    p.one_group = reinterpret_cast<int32_t*>(ws + L.one_group);
    p.n_tiles = p.one_group + 6;
    p.tiles = reinterpret_cast<Tile*>(ws + L.tiles);
    return p;
}

// launches a kernel of a call in turn behind the one before it on the stream
template <typename... P, typename... Q>
cudaError_t launch(void (*kern)(P...), dim3 grid, int block, size_t smem, cudaStream_t st, bool behind, Q... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, P(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_plan(const moe_adapter_params& p, const int32_t* ids, const Plan& plan, cudaStream_t st) {
    const size_t smem = (size_t)(34 * (p.n_adapters + 2)) * 4;
    cudaError_t e = allow_smem_once<adapter_plan_kernel>(34 * (kMaxAdapters + 2) * 4);
    if (e != cudaSuccess) return e;
    return launch(adapter_plan_kernel, dim3(1), 1024, smem, st, false, ids, (int)p.N, p.n_adapters, plan);
}

ShrinkArgs shrink_args(const moe_adapter_params& p, const void* X, const void* M, const float* scale, int K,
                       __nv_bfloat16* out, const Plan& plan) {
    ShrinkArgs a{};
    a.X = X;
    a.M = M;
    a.scale = scale;
    a.K = K;
    a.r = p.r;
    a.n_adapters = p.n_adapters;
    a.N = p.N;
    a.out = out;
    a.p = plan;
    return a;
}

// u, and v where it is given
template <typename T, int NQ>
cudaError_t launch_shrink_q(const moe_adapter_params& p, ShrinkArgs u, ShrinkArgs* v, cudaStream_t st) {
    constexpr size_t most_u = (size_t)kStages * shrink_stage<T, T, false>(NQ * 8),
                     most_v = (size_t)kStages * shrink_stage<T, float, true>(NQ * 8),
                     most_sums = (size_t)2 * kRows * NQ * 8 * 4;
    static_assert(std::max(most_u, most_v) <= 232448, "shared memory per CTA");
    size_t smem = std::max((size_t)kStages * shrink_stage<T, T, false>(p.r), (size_t)2 * kRows * p.r * 4);
    if (v) smem = std::max(smem, (size_t)kStages * shrink_stage<T, float, true>(p.r));
    cudaError_t e = v ? allow_smem_once<adapter_shrink_both_kernel<T, NQ>>(std::max({most_u, most_v, most_sums}))
                      : allow_smem_once<adapter_shrink_kernel<T, NQ>>(std::max(most_u, most_sums));
    if (e != cudaSuccess) return e;
    const int slices = shrink_slices(p, v ? std::max(u.K, v->K) : u.K, smem);
    auto cut = [&](int K) { return ((K + slices - 1) / slices + kShrinkK - 1) / kShrinkK * kShrinkK; };
    u.slice = cut(u.K);
    if (v) v->slice = cut(v->K);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tile_bound(p), (unsigned)slices, v ? 2 : 1);
    cfg.blockDim = dim3(kShrinkThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = (unsigned)slices;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = v ? cudaLaunchKernelEx(&cfg, adapter_shrink_both_kernel<T, NQ>, u, *v)
          : cudaLaunchKernelEx(&cfg, adapter_shrink_kernel<T, NQ>, u);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch_shrink(const moe_adapter_params& p, const ShrinkArgs& u, ShrinkArgs* v, cudaStream_t st) {
    if (p.r <= 16) return launch_shrink_q<T, 2>(p, u, v, st);
    if (p.r <= 32) return launch_shrink_q<T, 4>(p, u, v, st);
    if (p.r <= 64) return launch_shrink_q<T, 8>(p, u, v, st);
    return launch_shrink_q<T, 16>(p, u, v, st);
}

template <typename T, bool NN, int NK>
cudaError_t launch_expand_k(const moe_adapter_params& p, ExpandArgs a, bool behind, cudaStream_t st) {
    constexpr auto kern = adapter_expand_kernel<T, NN, NK>;
    // columns of a CTA: at most what leaves room for five CTAs on an SM, and few
    // enough that there are CTAs for two waves; more where the widest rows would
    // otherwise go in more spans than a grid has blocks in y
    const int64_t tiles = p.N / kRows + 1;
    auto smem = [](int span) { return (size_t)Parts<T>::self * expand_part<T, NN, NK>(span); };
    auto spans = [&](int span) { return ((int64_t)a.J + span - 1) / span; };
    static_assert((size_t)Parts<T>::self * expand_part<T, NN, NK>(256) <= 232448, "shared memory per CTA");
    static_assert(kMaxAdapterWidth / 256 <= 65535, "spans of the widest rows");
    a.span = 512;
    while (a.span > 128 && spans(a.span / 2) <= 65535 &&
           (smem(a.span) > 40 * 1024 || tiles * spans(a.span) < 2 * num_sms()))
        a.span /= 2;
    cudaError_t e = allow_smem_once<kern>(std::max(smem(256), (size_t)100 * 1024));
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)tile_bound(p), (unsigned)spans(a.span), 1);
    return launch(kern, grid, 128, smem(a.span), st, behind, a);
}

template <typename T, bool NN>
cudaError_t launch_expand(const moe_adapter_params& p, const __nv_bfloat16* in, const T* M, int J, const float* base,
                          float* out, int add_out, const Plan& plan, cudaStream_t st) {
    ExpandArgs a{};
    a.in = in;
    a.M = M;
    // behind a projection, whose kernel does not say when it may be followed, an ordinary launch
    a.base = add_out ? out : base;
    a.base2 = add_out ? base : nullptr;
    a.out = out;
    a.J = J;
    a.r = p.r;
    a.n_adapters = p.n_adapters;
    a.N = p.N;
    a.p = plan;
    if (p.r <= 16) return launch_expand_k<T, NN, 1>(p, a, !add_out, st);
    if (p.r <= 32) return launch_expand_k<T, NN, 2>(p, a, !add_out, st);
    if (p.r <= 64) return launch_expand_k<T, NN, 4>(p, a, !add_out, st);
    return launch_expand_k<T, NN, 8>(p, a, !add_out, st);
}

template <typename T, int MT>
cudaError_t launch_grads_m(const GradArgs& dA, const GradArgs& dB, cudaStream_t st) {
    constexpr auto kern = adapter_grad_kernel<T, MT>;
    constexpr size_t smem = grad_smem<Parts<T>::f32, MT>();
    static_assert(smem <= 232448, "shared memory per CTA");
    cudaError_t e = allow_smem_once<kern>(smem);
    if (e != cudaSuccess) return e;
    const int64_t ctas = (int64_t)((dA.J + kGradCols - 1) / kGradCols) * dA.ranges +
                         (int64_t)((dB.J + kGradCols - 1) / kGradCols) * dB.ranges;
    return launch(kern, dim3((unsigned)ctas), 128, smem, st, true, dA, dB);
}

template <typename T>
cudaError_t launch_grads(const moe_adapter_params& p, const __nv_bfloat16* u, const __nv_bfloat16* v, const T* x,
                         const float* dy, float* dA_out, float* dB_out, float* part_a, float* part_b, const Plan& plan,
                         cudaStream_t st) {
    GradArgs dA{};
    dA.in = v;
    dA.Z = x;
    dA.out = dA_out;
    dA.part = part_a;
    dA.J = p.d_in;
    dA.r = p.r;
    dA.n_adapters = p.n_adapters;
    dA.N = p.N;
    dA.p = plan;
    GradArgs dB = dA;
    dB.in = u;
    dB.Z = dy;
    dB.out = dB_out;
    dB.part = part_b;
    dB.J = p.d_out;
    grad_ranges(p, dA.ranges, dB.ranges);
    cudaError_t e = p.r <= 16   ? launch_grads_m<T, 1>(dA, dB, st)
                    : p.r <= 32 ? launch_grads_m<T, 2>(dA, dB, st)
                    : p.r <= 64 ? launch_grads_m<T, 4>(dA, dB, st)
                                : launch_grads_m<T, 8>(dA, dB, st);
    if (e != cudaSuccess) return e;
    // a CTA for 1024 of an adapter's elements, fewer where there are many adapters
    const int64_t n4 = (int64_t)p.r * std::max(p.d_in, p.d_out) / 4;
    const int64_t blocks = std::min<int64_t>((n4 + 255) / 256, std::max<int64_t>(1, 4 * (int64_t)num_sms() / p.n_adapters));
    return launch(adapter_reduce_kernel, dim3((unsigned)blocks, (unsigned)p.n_adapters, 2), 256, 0, st, true, dA, dB);
}

template <typename T>
cudaError_t forward(const moe_adapter_params& p, const T* x, const T* W, const T* A, const T* B, const float* scale,
                    const int32_t* ids, const float* base, float* y, char* ws, cudaStream_t st) {
    const Layout L = layout_of(p, W != nullptr, false);
    const Plan plan = plan_of(L, ws);
    const bool few = takes_tokens(p);
    const int slices = few_slices(p.N, p.d_in);
    float* part = reinterpret_cast<float*>(ws + L.u);
    __nv_bfloat16* u = reinterpret_cast<__nv_bfloat16*>(ws + L.u);
    cudaError_t e;
    if (few) {
        const int slice = ((p.d_in + slices - 1) / slices + 7) / 8 * 8;
        adapter_few_shrink_kernel<T><<<dim3(slices, (unsigned)p.N), 128, 0, st>>>(
            x, A, ids, (int)p.N, p.d_in, p.r, p.n_adapters, slice, part, plan.counters);
        e = cudaGetLastError();
    } else {
        e = launch_plan(p, ids, plan, st);
        if (e == cudaSuccess) e = launch_shrink<T>(p, shrink_args(p, x, A, scale, p.d_in, u, plan), nullptr, st);
    }
    if (e != cudaSuccess) return e;
    if (W) {
        int status = MOE_OK;
        moe_params q{};  // the projection as a layer of one expert with these rows
        q.N = p.N;
        q.d = p.d_out;
        q.d_f = p.d_in;
        q.E_r = 1;
        q.k = 1;
        q.dtype = p.dtype;
        if (sizeof(T) == 2 && !few && tc_tile_rows(q) == 256) {
            // enough rows for CTA pairs: 4096 x 4096 x 4096 in 102 us instead of 114 by single CTAs
            const ExpertWeights E{nullptr, nullptr, W, nullptr, nullptr, nullptr};
            e = launch_tc_down(q, DOWN_STORE, p.N, x, nullptr, plan.one_group, plan.one_group + 4, E, nullptr, nullptr,
                               nullptr, y, plan.counters, st, &status);
        } else if (sizeof(T) == 2) e = launch_tc_dense(p.N, p.d_out, p.d_in, x, W, y, plan.counters, st, &status);
        else
            e = launch_simt_dense(p.N, p.d_out, p.d_in, reinterpret_cast<const float*>(x), p.d_in, 1,
                                  reinterpret_cast<const float*>(W), p.d_in, 1, y, p.d_out, st);
        if (e != cudaSuccess) return e;
    }
    if (!few) return launch_expand<T, false>(p, u, B, p.d_out, base, y, W != nullptr, plan, st);
    return launch(adapter_few_expand_kernel<T>, dim3((unsigned)((p.d_out + 127) / 128), (unsigned)p.N), 128, 0, st, !W,
                  (const float*)part, slices, B, scale, ids, (int)p.N, p.d_out, p.r, p.n_adapters, base, y,
                  (int)(W != nullptr), plan.counters);
}

template <typename T>
cudaError_t backward(const moe_adapter_params& p, const T* x, const T* W, const T* A, const T* B, const float* scale,
                     const int32_t* ids, const float* dy, const float* dx_base, float* dx, float* dA, float* dB,
                     char* ws, cudaStream_t st) {
    const Layout L = layout_of(p, W != nullptr, true);
    const Plan plan = plan_of(L, ws);
    __nv_bfloat16* u = reinterpret_cast<__nv_bfloat16*>(ws + L.u);
    __nv_bfloat16* v = reinterpret_cast<__nv_bfloat16*>(ws + L.v);
    cudaError_t e = launch_plan(p, ids, plan, st);
    ShrinkArgs sv = shrink_args(p, dy, B, scale, p.d_out, v, plan);
    if (e == cudaSuccess) e = launch_shrink<T>(p, shrink_args(p, x, A, scale, p.d_in, u, plan), &sv, st);
    if (e != cudaSuccess) return e;
    if (W && sizeof(T) == 2) {
        __nv_bfloat16* hi = reinterpret_cast<__nv_bfloat16*>(ws + L.hi);
        __nv_bfloat16* lo = reinterpret_cast<__nv_bfloat16*>(ws + L.lo);
        const int64_t n = p.N * (int64_t)p.d_out;
        e = launch(adapter_split_kernel, dim3((unsigned)min64((n / 8 + 255) / 256, (int64_t)num_sms() * 8)), 256, 0, st,
                   true, dy, n, hi, lo);
        if (e != cudaSuccess) return e;
        moe_params q{};
        q.N = p.N;
        q.E_r = 1;
        q.k = 1;
        q.dtype = MOE_BF16;
        int status = MOE_OK;
        // the small parts' products first: behind the large ones' sum each of their additions
        // would be cut off at its size (4096 tokens, 4096 to 4096: dx 1.3e-5 of its norm off).
        // Few output tiles: K is split over CTAs, which add into dx (139 tokens, 1432 x 2608: 100 -> 70 us)
        const bool split_k = tc_store_bmn_split(q, p.d_in, p.d_out, true) > 1;
        if (split_k && (e = cudaMemsetAsync(dx, 0, sizeof(float) * p.N * p.d_in, st)) != cudaSuccess) return e;
        e = launch_tc_store_bmn(q, p.d_in, p.d_out, lo, p.d_out, W, hi, p.d_out, W, plan.one_group, plan.one_group + 2,
                                dx, plan.counters, st, &status, split_k);
    } else if (W) {
        e = launch_simt_dense(p.N, p.d_in, p.d_out, dy, p.d_out, 1, reinterpret_cast<const float*>(W), 1, p.d_in, dx,
                              p.d_in, st);
    }
    if (e == cudaSuccess) e = launch_expand<T, true>(p, v, A, p.d_in, dx_base, dx, W != nullptr, plan, st);
    if (e == cudaSuccess) e = launch_grads<T>(p, u, v, x, dy, dA, dB, reinterpret_cast<float*>(ws + L.part_a),
                                            reinterpret_cast<float*>(ws + L.part_b), plan, st);
    return e;
}

// what a call with a projection needs besides
moe_status check_projection(const moe_adapter_params* p, const void* W) {
    if (W && p->dtype == MOE_F32 && p->N > (int64_t)65535 * 64) {
        record_error("moe_adapter: at most 65535 * 64 tokens through an fp32 projection");
        return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

moe_status check(const moe_adapter_params* p) {
    if (!p) return MOE_ERR_INVALID_ARG;
    if (p->N < 0 || p->d_in < 1 || p->d_out < 1 || p->n_adapters < 1 || p->r < 1) return MOE_ERR_INVALID_ARG;
    if (p->dtype != MOE_F32 && p->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (p->d_in % 8 || p->d_out % 8 || p->r % 8) {
        record_error("moe_adapter: d_in, d_out and r must be multiples of 8");
        return MOE_ERR_UNSUPPORTED;
    }
    if (p->r > kMaxAdapterRank || p->n_adapters > kMaxAdapters || p->N >= (int64_t)1 << 30 || p->d_in > kMaxAdapterWidth ||
        p->d_out > kMaxAdapterWidth) {
        record_error("moe_adapter: at most rank 128, 1024 adapters, 2^30 - 1 tokens and widths of 2^23");
        return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_adapter_workspace_size(const moe_adapter_params* p, int with_W, size_t* bytes) {
    const moe_status s = check(p);
    if (s != MOE_OK) return s;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = layout_of(*p, with_W != 0, false).total;
    return MOE_OK;
}

moe_status moe_adapter_backward_workspace_size(const moe_adapter_params* p, int with_W, size_t* bytes) {
    const moe_status s = check(p);
    if (s != MOE_OK) return s;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = layout_of(*p, with_W != 0, true).total;
    return MOE_OK;
}

moe_status moe_adapter_forward(const moe_adapter_params* p, const void* x, const void* W, const void* A, const void* B,
                               const float* scale, const int32_t* ids, const float* base, float* y, void* ws,
                               moe_stream_t stream) {
    moe_status s = check(p);
    if (s == MOE_OK) s = check_projection(p, W);
    if (s != MOE_OK) return s;
    if (!ws || !aligned16(ws)) return MOE_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    (void)cudaGetLastError();
    char* w = static_cast<char*>(ws);
    if (p->N == 0)
        return cuda_status(cudaMemsetAsync(w + layout_of(*p, false, false).counters, 0, CNT_COUNT * 8, st),
                         "moe_adapter_forward memset");
    if (!x || !A || !B || !scale || !ids || !y) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(W) || !aligned16(A) || !aligned16(B) || !aligned16(base) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
    if (W && base == y) return MOE_ERR_INVALID_ARG;  // the projection is written before base is added
    const cudaError_t e =
        p->dtype == MOE_BF16
            ? forward(*p, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(W),
                      static_cast<const __nv_bfloat16*>(A), static_cast<const __nv_bfloat16*>(B), scale, ids, base, y, w, st)
            : forward(*p, static_cast<const float*>(x), static_cast<const float*>(W), static_cast<const float*>(A),
                      static_cast<const float*>(B), scale, ids, base, y, w, st);
    return cuda_status(e, "moe_adapter_forward");
}

moe_status moe_adapter_backward(const moe_adapter_params* p, const void* x, const void* W, const void* A, const void* B,
                                const float* scale, const int32_t* ids, const float* dy, const float* dx_base,
                                float* dx, float* dA, float* dB, void* ws, moe_stream_t stream) {
    moe_status s = check(p);
    if (s == MOE_OK) s = check_projection(p, W);
    if (s != MOE_OK) return s;
    if (!ws || !aligned16(ws)) return MOE_ERR_WORKSPACE;
    if (!dA || !dB || !aligned16(dA) || !aligned16(dB)) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    (void)cudaGetLastError();
    char* w = static_cast<char*>(ws);
    if (p->N == 0) {
        const size_t n = (size_t)p->n_adapters * p->r * 4;
        cudaError_t e = cudaMemsetAsync(w + layout_of(*p, false, true).counters, 0, CNT_COUNT * 8, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dA, 0, n * p->d_in, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dB, 0, n * p->d_out, st);
        return cuda_status(e, "moe_adapter_backward memset");
    }
    if (!x || !A || !B || !scale || !ids || !dy || !dx) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(W) || !aligned16(A) || !aligned16(B) || !aligned16(dy) || !aligned16(dx_base) || !aligned16(dx))
        return MOE_ERR_INVALID_ARG;
    if (W && dx_base == dx) return MOE_ERR_INVALID_ARG;
    const cudaError_t e =
        p->dtype == MOE_BF16
            ? backward(*p, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(W),
                       static_cast<const __nv_bfloat16*>(A), static_cast<const __nv_bfloat16*>(B), scale, ids, dy,
                       dx_base, dx, dA, dB, w, st)
            : backward(*p, static_cast<const float*>(x), static_cast<const float*>(W), static_cast<const float*>(A),
                       static_cast<const float*>(B), scale, ids, dy, dx_base, dx, dA, dB, w, st);
    return cuda_status(e, "moe_adapter_backward");
}

moe_status moe_adapter_check(const moe_adapter_params* p, const void* ws, moe_stream_t stream) {
    const moe_status s = check(p);
    if (s != MOE_OK) return s;
    if (!ws) return MOE_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    unsigned long long cnt[CNT_COUNT];
    cudaError_t e = cudaMemcpyAsync(cnt, static_cast<const char*>(ws) + layout_of(*p, false, false).counters,
                                    sizeof(cnt), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return cuda_status(e, "moe_adapter_check");
    if (cnt[CNT_DEVICE_ERROR] & DEVERR_TIMEOUT) return MOE_ERR_TIMEOUT;
    if (cnt[CNT_DEVICE_ERROR] & DEVERR_BOUNDS) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // extern "C"
