// rowring.cuh -- the bulk-copy ring of the residual-stream kernels, and the
// vectors of their rows.
//
// A CTA takes row blocks b = blockIdx.x, + gridDim.x, ... of R rows; each
// input's block is one bulk copy (rows in order) or one copy a row (rows
// placed by a RowMap).  Unlike the ring of common.cuh, the inputs may have
// different row lengths (an 8-bit checkpoint beside 16-bit gradients) and
// rows of any length: a block that does not start or end on a 16-byte
// boundary is copied from the boundary below to the one above it, clipped to
// the input's whole 16-byte units; what lies past those (the input's last 15
// bytes at most) the last block's threads put into the slot themselves.
//
// Vectors.  A row of N elements starts at element r N of a contiguous tensor.
// The vectors are those of the storage: VEC elements from a multiple of VEC
// on, so they are aligned in every tensor of [M, N] whatever its element
// size, and a row whose length is no multiple of VEC has partial vectors at
// its ends (kEdge): the elements of other rows in them are masked.  CTAs
// step by a multiple of VEC rows, so a thread's mask and its weights stay
// the same over all of its rows.
#pragma once

#include "addnorm.cuh"

namespace gbn {

// Schedules.  A row of up to `cap` vectors goes to a row group of W threads
// with KV vectors each (vector v of the row to thread v % W); a CTA of T
// threads has G = T / W groups.  Up to 32 vectors: one a lane.  From there on
// several a thread, which then share the row's reduction, its barrier and the
// ring's work.  A warp skips those of its KV vectors that lie past the row's
// end.  Rows that leave many lanes of a fixed group idle (kRowFit) take groups
// of as many warps as they fill.
//   Two vectors (kRow2): the forwards that write as many 16-bit values as they
// read, and the backwards, which hold a column sum and a weight of every
// element next to the row.  What bounds y is how many copies are in flight:
// with two CTAs of two 16 KB stages an SM, 64 KB, N = 1024 runs at 94% of the
// copy rate, with 128 KB at 88%.
//   Four (kRow4, and kRow2 from kRowMore on): the 8-bit output and the
// checkpoint alone, which write less and compute more (8-bit output N = 2048:
// 92%, with two vectors 85%); rows that do not fill their group; and the
// backward from a checkpoint.  A backward with four reads its row from the
// ring a second time instead of keeping it (128 registers hold the sums, the
// weights and little more).
struct RowSched {
    int cap, W, KV, T;  // W 0: kRowFit, chosen in the launch
};
constexpr int kNumRowSched = 16, kRowFit = 10, kRowFit2 = 11, kRowMore = 12;
constexpr RowSched kRow2[kNumRowSched] = {  // 9 and kRowFit: four
    {4, 4, 1, 256},      {8, 8, 1, 256},      {16, 16, 1, 256},   {32, 32, 1, 256},
    {64, 32, 2, 256},    {128, 64, 2, 256},   {256, 128, 2, 256}, {512, 256, 2, 256},
    {1024, 512, 2, 512}, {2048, 512, 4, 512}, {1024, 0, 4, 256},  {512, 0, 2, 256},
    {128, 32, 4, 256},   {256, 64, 4, 256},   {512, 128, 4, 256}, {1024, 256, 4, 256},
};
constexpr RowSched kRow4[kNumRowSched] = {
    {4, 4, 1, 256},      {8, 8, 1, 256},      {16, 16, 1, 256},  {32, 32, 1, 256},
    {64, 32, 2, 256},    {128, 32, 4, 256},   {256, 64, 4, 256}, {512, 128, 4, 256},
    {1024, 256, 4, 256}, {2048, 512, 4, 512}, {1024, 0, 4, 256}, {512, 0, 2, 256},
};
// Kinds of kernels: 8-bit output or checkpoint alone; y (and checkpoint); backward.
enum RowKind : int { kKindQ = 0, kKindY = 1, kKindB = 2 };
// Whether kernels of a kind take schedule S (the others are not built).
constexpr bool row_takes(int kind, int S)
{
    return S <= kRowFit || (S == kRowFit2 ? kind != kKindY : kind != kKindQ);
}
constexpr int fwd_kind(int mode)
{
    return (mode & 3) == kModeY || (mode & 3) == kModeYC ? kKindY : kKindQ;
}
constexpr const RowSched& row_sched(int kind, int S)
{
    return kind == kKindQ ? kRow4[S] : kRow2[S];
}
// Row groups of a CTA (kRowFit: with W threads each).
constexpr int row_G(int kind, int S, int W = 0)
{
    const RowSched& e = row_sched(kind, S);
    return e.W ? e.T / e.W : W <= 64 ? 4 : W <= 128 ? 2 : 1;
}
// Rows a thread takes of a block: two of one vector.  (A thread's rows of a
// block are G apart, a multiple of VEC: rows that start inside a vector keep
// one mask and one set of weights a thread.)
constexpr int row_U(int kind, int S) { return row_sched(kind, S).KV == 1 ? 2 : 1; }
// CTAs an SM holds at least (their register budget), and ring stages.
constexpr int row_minb(int kind, int S)
{
    const RowSched& e = row_sched(kind, S);
    if (e.T == 512) return 1;
    return kind != kKindB && (e.KV == 1 || (e.KV == 2 && kind == kKindQ)) ? 3 : 2;
}
constexpr int row_stages(int kind, int S)
{
    return kind == kKindB && row_sched(kind, S).KV < 4 ? 3 : 2;
}
// Dynamic shared memory the kernels may ask for: three inputs of the widest
// rows (32 KB each) in two stages, and room for the group maxima.
constexpr int kMaxSmem = 208 * 1024;

#ifdef __CUDACC__

// ------------------------------------------------------------------ ring
// Block b into stage st: every lane of warp 0.  Lane t takes input t (the
// barrier counts an arrival per input), so a block costs one input's
// arithmetic: the other warps meet this one at every row's barrier, and
// taking the inputs one after another on one lane cost the backwards 5-25%.
template <int NT>
__device__ __forceinline__ void row_issue(const RowSrc (&in)[NT], const RowPlan& pl, int64_t M,
                                          unsigned char* dsm, int64_t b, int st)
{
    uint64_t* const bar = reinterpret_cast<uint64_t*>(dsm) + st;
    unsigned char* const slot = dsm + 128 + (size_t)st * pl.stage_bytes;
    const int lane = threadIdx.x & 31;
    const int64_t r0 = b * pl.R;
    // lane t's input (selects: indexing the parameters would copy them)
    const unsigned char* p = nullptr;
    uint32_t rb = 0, off = 0;
    int64_t total = 0;
    int scattered = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t)
        if (lane == t) {
            p = in[t].p;
            rb = (uint32_t)in[t].row_bytes;
            total = in[t].total;
            scattered = in[t].scattered;
            off = pl.off[t];
        }
    if (p) {
        const bool last = b == pl.nblocks - 1;
        if (scattered) {
            mbar_expect_tx(bar, (uint32_t)(last ? (int)(M - r0) : pl.R) * rb);
        } else {
            // from the 16-byte boundary below the block to the one above it;
            // the last block's end is clipped to the input's whole units
            const uint32_t rows = (uint32_t)pl.R * rb;
            const int64_t at = b * (int64_t)rows;
            const uint32_t low = (uint32_t)at & 15u;
            uint32_t n = (low + rows + 15u) & ~15u;
            if (last) n = (uint32_t)((total & ~(int64_t)15) - (at - low));
            mbar_expect_tx(bar, n);
            if (n) bulk_g2s(slot + off, p + (at - low), n, bar);
        }
    }
    if (!pl.in_order) {
        const int rows = (int)(M - r0 < pl.R ? M - r0 : pl.R);
        __syncwarp();  // the expected bytes are set before a copy lands
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (in[t].p && in[t].scattered)
                for (int i = lane; i < rows; i += 32)
                    bulk_g2s(slot + pl.off[t] + i * (uint32_t)in[t].row_bytes,
                             in[t].p + row_byte_offset(in[t].map, r0 + i),
                             (uint32_t)in[t].row_bytes, bar);
    }
}

// The bytes of block b past the inputs' whole 16-byte units, into the slot:
// every thread, once the block's copies have landed; the caller synchronizes.
template <int NT>
__device__ __noinline__ void row_tail(const RowSrc (&in)[NT], const RowPlan& pl,
                                      unsigned char* slot, int64_t b)
{
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (!in[t].p || in[t].scattered) continue;
        const int64_t start = (b * pl.R * in[t].row_bytes) & ~(int64_t)15;
        const int64_t i = (in[t].total & ~(int64_t)15) + threadIdx.x;
        if (i < in[t].total) slot[pl.off[t] + (i - start)] = in[t].p[i];
    }
}

// Start the ring: the barriers, and the first blocks' copies.
template <int NT>
__device__ __forceinline__ int64_t row_ring_start(const RowSrc (&in)[NT], const RowPlan& pl,
                                                  int64_t M, unsigned char* dsm)
{
    const int64_t K = pl.nblocks > (int64_t)blockIdx.x
                          ? (pl.nblocks - 1 - blockIdx.x) / gridDim.x + 1
                          : 0;
    if (threadIdx.x == 0) {
        int n = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t) n += in[t].p != nullptr;
        for (int s = 0; s < pl.stages; ++s) mbar_init(reinterpret_cast<uint64_t*>(dsm) + s, n);
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x < 32)
        for (int k = 0; k < pl.stages && k < K; ++k)
            row_issue(in, pl, M, dsm, blockIdx.x + (int64_t)k * gridDim.x, k);
    return K;
}

// body(b, slot, alive) for each of the CTA's K blocks.  body returns true
// when it passed a __syncthreads after its last read of the slot (the same
// answer on every thread); otherwise the ring adds one.  A wait that runs out
// sets the fault word; the CTA then runs its remaining blocks without loads
// or stores and waits, bounded again, for its copies in flight.
template <int NT, class Body>
__device__ __forceinline__ void row_ring(const RowSrc (&in)[NT], const RowPlan& pl, int64_t M,
                                         unsigned char* dsm, int64_t K, Body&& body)
{
    uint64_t* const bar = reinterpret_cast<uint64_t*>(dsm);
    int st = 0;
    uint32_t phase = 0;
    bool alive = true;
    int64_t failed_at = K, b = blockIdx.x;
    for (int64_t k = 0; k < K; ++k) {
        unsigned char* const slot = dsm + 128 + (size_t)st * pl.stage_bytes;
        if (alive) {
            alive = mbar_wait(&bar[st], phase, pl.fault);
            if (!alive) failed_at = k;
        }
        if (pl.tail && b == pl.nblocks - 1) {  // uniform; a failed wait loads nothing below
            row_tail(in, pl, slot, b);
            __syncthreads();
        }
        if (!body(b, slot, alive)) __syncthreads();
        // one answer for warp 0: its lanes issue together
        if (threadIdx.x < 32 && __all_sync(0xffffffffu, alive) && k + pl.stages < K) {
            fence_proxy_async();
            row_issue(in, pl, M, dsm, b + (int64_t)pl.stages * gridDim.x, st);
        }
        b += gridDim.x;
        if (++st == pl.stages) {
            st = 0;
            phase ^= 1;
        }
    }
    if (!alive)
        for (int64_t k = failed_at; k < K && k < failed_at + pl.stages; ++k)
            mbar_wait(&bar[k % pl.stages], (uint32_t)((k / pl.stages) & 1), nullptr, kWaitCycles);
    __syncthreads();
}

// --------------------------------------------------------------- vectors
// Byte offset in the slot of the first element of row i of the block from row
// r0 on.  CTAs step by a multiple of VEC rows, so for rows of activations it
// is the same in every block of a CTA.
__device__ __forceinline__ uint32_t row_off(const RowSrc& s, int64_t r0, int i)
{
    const uint32_t rb = (uint32_t)s.row_bytes;
    return (s.scattered ? 0u : ((uint32_t)r0 * rb) & 15u) + (uint32_t)i * rb;
}

__device__ __forceinline__ uint2 lds64(const void* p)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(smem_u32(p)));
    return v;
}
__device__ __forceinline__ uint32_t lds32(const void* p)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)));
    return v;
}

// The NW words of a vector with the elements outside the mask zeroed.
template <int VEC, int NW>
__device__ __forceinline__ void mask_words(uint32_t (&v)[NW], uint32_t em)
{
    constexpr int per = VEC / NW, bits = 32 / per;  // elements a word
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
        for (int e = 0; e < per; ++e)
            if (!((em >> (i * per + e)) & 1u))
                v[i] &= per == 1 ? 0u : ~(((1u << (bits % 32)) - 1u) << (e * bits % 32));
}

// 16 bytes of activations at byte o of the slot; cut: masked.
template <typename TX>
__device__ __forceinline__ uint4 ld_vec(const unsigned char* slot, uint32_t o, bool ok, bool cut,
                                        uint32_t em)
{
    uint4 v = lds128_if(ok, slot + o);
    if (cut) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        mask_words<Vec<TX>::kN>(w, em);
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

// A vector's VEC 8-bit values.
template <int VEC>
__device__ __forceinline__ void ld_vec8(uint32_t (&v)[VEC / 4], const unsigned char* slot,
                                        uint32_t o, bool ok, bool cut, uint32_t em)
{
    if constexpr (VEC == 8) {
        const uint2 q = ok ? lds64(slot + o) : make_uint2(0, 0);
        v[0] = q.x;
        v[1] = q.y;
    } else {
        v[0] = ok ? lds32(slot + o) : 0u;
    }
    if (cut) mask_words<VEC>(v, em);
}

// Word p of a vector.
__device__ __forceinline__ uint32_t word(const uint4& v, int p)
{
    return p == 0 ? v.x : p == 1 ? v.y : p == 2 ? v.z : v.w;
}

// Store a vector of activations; cut: the elements in the mask.
template <typename TX>
__device__ __forceinline__ void st_vec(TX* p, const uint4& v, bool ok, bool cut, uint32_t em)
{
    constexpr uint32_t kFull = (1u << Vec<TX>::kN) - 1u;
    st_stream_if(ok && (!cut || em == kFull), p, v);
    if (cut && ok && em != kFull) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < Vec<TX>::kN; ++e)
            if ((em >> e) & 1u) {
                if constexpr (sizeof(TX) == 2)
                    reinterpret_cast<unsigned short*>(p)[e] =
                        (unsigned short)(w[e / 2] >> (16 * (e % 2)));
                else
                    reinterpret_cast<uint32_t*>(p)[e] = w[e];
            }
    }
}

template <int VEC>
__device__ __forceinline__ void st_vec8(unsigned char* p, const uint32_t (&v)[VEC / 4], bool ok,
                                        bool cut, uint32_t em)
{
    constexpr uint32_t kFull = (1u << VEC) - 1u;
    if (ok && (!cut || em == kFull)) {
        if constexpr (VEC == 8)
            __stcs(reinterpret_cast<uint2*>(p), make_uint2(v[0], v[1]));
        else
            __stcs(reinterpret_cast<unsigned*>(p), v[0]);
    }
    if (cut && ok && em != kFull) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if ((em >> e) & 1u) p[e] = (unsigned char)(v[e / 4] >> (8 * (e % 4)));
    }
}

// A thread's part of its rows: its vector j is vector l + j W of the row,
// whose element 0 is column col(j) = (l + j W) VEC - first, and em[j] says
// which of its elements are the row's.  The first `live` of them have a lane
// of this warp in the row.
template <int VEC, int kW, int KV, bool kEdge>
struct Cols {
    int l, W, first, live;
    uint32_t em[KV];
    uint32_t partial;  // bit j: a lane of this warp holds part of a vector j (the same on all)
    __device__ Cols(int lane, int W_, int first_, int N)
        : l(lane), W(kW ? kW : W_), first(kEdge ? first_ : 0), live(0)
    {
#pragma unroll
        for (int j = 0; j < KV; ++j) {
            const int c = col(j), lo = c < 0 ? -c : 0, hi = N - c < VEC ? N - c : VEC;
            em[j] = hi > lo ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
            if (KV == 1 || c - (l & 31) * VEC < N) live = j + 1;
        }
        partial = 0;
        if constexpr (kEdge) {
#pragma unroll
            for (int j = 0; j < KV; ++j)
                if (__any_sync(0xffffffffu, em[j] != 0 && em[j] != (1u << VEC) - 1u))
                    partial |= 1u << j;
        }
    }
    __device__ int vec(int j) const { return l + j * W; }
    __device__ int col(int j) const { return vec(j) * VEC - first; }
    __device__ bool ok(int j) const { return em[j] != 0; }
    // Whether vector j of some lane is partial: only then are loads masked and
    // stores split (a warp-uniform branch).
    __device__ bool cut(int j) const { return kEdge && ((partial >> j) & 1u); }
};

// Weights of a thread's vectors as float32 (1 + w for Gemma), zeros outside
// the row.  Whole vectors of an aligned weight come as 16-byte loads.
template <int VEC, int kW, int KV, bool kEdge>
__device__ __forceinline__ void load_weights(f2 (&wf)[KV][VEC / 2],
                                             const Cols<VEC, kW, KV, kEdge>& c,
                                             const void* w, int wt, bool gemma)
{
    constexpr int P = VEC / 2;
    const f2 one = splat2(gemma ? 1.f : 0.f);
    if (!kEdge && (reinterpret_cast<uintptr_t>(w) & 15) == 0 && (VEC == 8 || wt == kF32)) {
#pragma unroll
        for (int j = 0; j < KV; ++j) {
#pragma unroll
            for (int p = 0; p < P; ++p) wf[j][p] = splat2(0.f);
            if (!c.ok(j)) continue;
            if (wt == kF32) {
#pragma unroll
                for (int q = 0; q < P / 2; ++q) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(
                        static_cast<const float*>(w) + c.col(j) + 4 * q));
                    wf[j][2 * q] = mk2(v.x, v.y);
                    wf[j][2 * q + 1] = mk2(v.z, v.w);
                }
            } else if constexpr (VEC == 8) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(
                    static_cast<const unsigned short*>(w) + c.col(j)));
                if (wt == kBF16)
                    unpack2<__nv_bfloat16>(v, wf[j]);
                else
                    unpack2<__half>(v, wf[j]);
            }
#pragma unroll
            for (int p = 0; p < P; ++p) wf[j][p] = add2(wf[j][p], one);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < KV; ++j)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = (c.em[j] >> (2 * p + h)) & 1u;
                v[h] = in ? ld_param(w, wt, c.col(j) + 2 * p + h) + (gemma ? 1.f : 0.f) : 0.f;
            }
            wf[j][p] = mk2(v[0], v[1]);
        }
}

// Sums (and NaN-keeping maxima) over the threads of a row group, U rows at
// once: every thread of a group gets the same bits.  kLanes <= 32: a group is
// kLanes lanes of a warp.  Otherwise it is up to kLanes / 32 whole warps,
// joined through `red` (row_red_floats; zero where no warp writes) with one
// __syncthreads; its two halves are used in turn.
template <int kLanes, int G, int U, bool kMax>
__device__ __forceinline__ void row_reduce(float (&s)[U], float (&m)[U], float* red, int& parity,
                                           int g, int l)
{
    constexpr int kIn = kLanes < 32 ? kLanes : 32;
    butterfly<kIn, U>(s);
    if constexpr (kMax) {
#pragma unroll
        for (int off = kIn / 2; off >= 1; off >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u)
                m[u] = max_nan(m[u], __shfl_xor_sync(0xffffffffu, m[u], off));
    }
    if constexpr (kLanes > 32) {
        constexpr int kWarps = kLanes / 32, kV = kMax ? 2 * U : U;
        const int lane = threadIdx.x & 31;
        float* slot = red + (parity * G + g) * kV * kWarps;
        if (lane == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                slot[u * kWarps + (l >> 5)] = s[u];
                if constexpr (kMax) slot[(U + u) * kWarps + (l >> 5)] = m[u];
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = slot[u * kWarps + (lane & (kWarps - 1))];
            if constexpr (kMax) m[u] = slot[(U + u) * kWarps + (lane & (kWarps - 1))];
        }
        butterfly<kWarps, U>(s);
        if constexpr (kMax) {
#pragma unroll
            for (int off = kWarps / 2; off >= 1; off >>= 1)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    m[u] = max_nan(m[u], __shfl_xor_sync(0xffffffffu, m[u], off));
        }
        parity ^= 1;
    }
}
template <int kLanes, int G, int U, bool kMax>
constexpr int row_red_floats()
{
    return kLanes > 32 ? 2 * G * (kMax ? 2 * U : U) * (kLanes / 32) : 1;
}

// Largest magnitude of a vector's elements, NaN on top, from its packed form:
// 16-bit types compare in pairs (exact).
template <typename TX>
__device__ __forceinline__ float vec_amax(const uint4& v)
{
    if constexpr (is16<TX>()) {
        constexpr uint32_t kAbs = 0x7fff7fffu;
        const uint32_t w[4] = {v.x & kAbs, v.y & kAbs, v.z & kAbs, v.w & kAbs};
        uint32_t a, b, r;
        if constexpr (std::is_same<TX, __half>::value) {
            asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(a) : "r"(w[0]), "r"(w[1]));
            asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(b) : "r"(w[2]), "r"(w[3]));
            asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        } else {
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w[0]), "r"(w[1]));
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w[2]), "r"(w[3]));
            asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        }
        const f2 f = P16<TX>::to_f2(r);
        return max_nan(lo2(f), hi2(f));
    } else {
        f2 p[2];
        unpack2<TX>(v, p);
        return max_nan(max_nan(fabsf(lo2(p[0])), fabsf(hi2(p[0]))),
                       max_nan(fabsf(lo2(p[1])), fabsf(hi2(p[1]))));
    }
}

// f(std::integral_constant<int, S>) for schedule sid.
template <class F>
inline bool with_row_sched(int sid, F&& f)
{
    switch (sid) {
        case 0: f(std::integral_constant<int, 0>{}); return true;
        case 1: f(std::integral_constant<int, 1>{}); return true;
        case 2: f(std::integral_constant<int, 2>{}); return true;
        case 3: f(std::integral_constant<int, 3>{}); return true;
        case 4: f(std::integral_constant<int, 4>{}); return true;
        case 5: f(std::integral_constant<int, 5>{}); return true;
        case 6: f(std::integral_constant<int, 6>{}); return true;
        case 7: f(std::integral_constant<int, 7>{}); return true;
        case 8: f(std::integral_constant<int, 8>{}); return true;
        case 9: f(std::integral_constant<int, 9>{}); return true;
        case 10: f(std::integral_constant<int, 10>{}); return true;
        case 11: f(std::integral_constant<int, 11>{}); return true;
        case 12: f(std::integral_constant<int, 12>{}); return true;
        case 13: f(std::integral_constant<int, 13>{}); return true;
        case 14: f(std::integral_constant<int, 14>{}); return true;
        case 15: f(std::integral_constant<int, 15>{}); return true;
        default: return false;
    }
}

#endif  // __CUDACC__

}  // namespace gbn
