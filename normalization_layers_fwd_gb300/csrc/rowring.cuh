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
// bytes at most) is read from global memory by the last block.
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

// Schedules.  A row of nvec vectors goes to a row group of W threads with KV
// vectors each (vector v of the row to thread v % W); a CTA has G groups.  Up
// to 64 vectors a group is (part of) a warp, with W the next power of two;
// wider rows take as many warps as they fill, W = 32 ceil(nvec / (32 KV)), so
// that no more than a warp's worth of lanes idles.  Two vectors a thread
// halve the reduction that one would take.  The widest backward holds its
// column sums and weights in registers (T <= 512 leaves 128 each) and reads
// its row from the ring once more instead of keeping it (row_lean).
struct RowSched {
    int cap, W, G, KV, T;  // W 0: as many warps as the row fills, T / G threads at most
};
constexpr int kNumRowSched = 10;
constexpr RowSched kRowFwd[kNumRowSched] = {
    {4, 4, 64, 1, 256},    {8, 8, 32, 1, 256},   {16, 16, 16, 1, 256}, {32, 32, 8, 1, 256},
    {64, 32, 8, 2, 256},   {128, 0, 4, 2, 256},  {256, 0, 2, 2, 256},  {512, 0, 1, 2, 256},
    {1024, 0, 1, 2, 512},  {2048, 0, 1, 2, 1024},
};
constexpr RowSched kRowBwd[kNumRowSched] = {
    {4, 4, 64, 1, 256},    {8, 8, 32, 1, 256},   {16, 16, 16, 1, 256}, {32, 32, 8, 1, 256},
    {64, 32, 8, 2, 256},   {128, 0, 4, 2, 256},  {256, 0, 2, 2, 256},  {512, 0, 1, 2, 256},
    {1024, 0, 1, 2, 512},  {2048, 0, 1, 4, 512},
};
constexpr const RowSched& row_sched(bool bwd, int S) { return bwd ? kRowBwd[S] : kRowFwd[S]; }
constexpr int row_W(bool bwd, int S, int64_t nvec)
{
    const RowSched& e = row_sched(bwd, S);
    return e.W ? e.W : (int)((nvec + 32 * e.KV - 1) / (32 * e.KV)) * 32;
}
constexpr bool row_lean(int S) { return S == 9; }
#ifndef GBN_FU
#define GBN_FU 1
#endif
#ifndef GBN_BU
#define GBN_BU 1
#endif
// Rows a thread takes of a block.  Rows that start inside a vector keep one
// mask and one set of weights a thread, so a thread's rows of a block are a
// multiple of VEC rows apart (G) or one.
constexpr int row_U(bool bwd, int S, bool edge)
{
    const RowSched& e = row_sched(bwd, S);
    return e.KV == 1 ? 2 : e.T > 512 || e.KV > 2 || (edge && e.G % 8 != 0) ? 1
           : bwd ? GBN_BU : GBN_FU;
}
constexpr int row_R(bool bwd, int S, bool edge)
{
    return row_sched(bwd, S).G * row_U(bwd, S, edge);
}
// CTAs of T threads an SM holds at least (their register budget), and ring
// stages.
#ifndef GBN_FMINB
#define GBN_FMINB 3
#endif
#ifndef GBN_FST
#define GBN_FST 2
#endif
#ifndef GBN_BMINB
#define GBN_BMINB 2
#endif
#ifndef GBN_BST
#define GBN_BST 3
#endif
constexpr int fwd_minb(int S, bool edge)
{
    const RowSched& e = kRowFwd[S];
    return e.T == 256 ? (e.KV == 1 && !edge ? 4 : GBN_FMINB) : e.T == 512 && !edge ? 2 : 1;
}
constexpr int bwd_minb(int S) { return kRowBwd[S].T == 256 ? GBN_BMINB : 1; }
constexpr int fwd_stages(int S) { return kRowFwd[S].T == 256 ? GBN_FST : 3; }
constexpr int bwd_stages(int S) { return S == 9 ? 2 : GBN_BST; }
// Registers a thread may use, from the CTAs asked for.
constexpr int row_regs(int T, int minb) { return 65536 / (T * minb) / 8 * 8; }
// Dynamic shared memory the kernels may ask for: three inputs of the widest
// rows (32 KB each) in two stages, and room for the group maxima.
constexpr int kMaxSmem = 208 * 1024;

#ifdef __CUDACC__

// ------------------------------------------------------------------ ring
// Block b into stage st: every lane of warp 0.
template <int NT>
__device__ __forceinline__ void row_issue(const RowSrc (&in)[NT], const RowPlan& pl, int64_t M,
                                          unsigned char* dsm, int64_t b, int st)
{
    uint64_t* const bar = reinterpret_cast<uint64_t*>(dsm) + st;
    unsigned char* const slot = dsm + 128 + (size_t)st * pl.stage_bytes;
    const int lane = threadIdx.x & 31;
    const int64_t r0 = b * pl.R;
    const int rows = (int)(M - r0 < pl.R ? M - r0 : pl.R);
    int64_t start[NT];
    uint32_t n[NT], sum = 0;
    bool scattered = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        n[t] = 0;
        if (!in[t].p) continue;
        if (in[t].scattered) {
            scattered = true;
            n[t] = (uint32_t)(rows * in[t].row_bytes);
        } else {
            start[t] = (r0 * in[t].row_bytes) & ~(int64_t)15;
            int64_t end = ((r0 + rows) * in[t].row_bytes + 15) & ~(int64_t)15;
            const int64_t whole = in[t].total & ~(int64_t)15;
            end = end < whole ? end : whole;
            n[t] = end > start[t] ? (uint32_t)(end - start[t]) : 0;
        }
        sum += n[t];
    }
    if (lane == 0) {
        mbar_expect_tx(bar, sum);
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (n[t] && !in[t].scattered) bulk_g2s(slot + pl.off[t], in[t].p + start[t], n[t], bar);
    }
    if (scattered) {
        __syncwarp();  // the expected bytes are set before a copy lands
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (n[t] && in[t].scattered)
                for (int i = lane; i < rows; i += 32)
                    bulk_g2s(slot + pl.off[t] + i * (uint32_t)in[t].row_bytes,
                             in[t].p + row_byte_offset(in[t].map, r0 + i),
                             (uint32_t)in[t].row_bytes, bar);
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
        for (int s = 0; s < pl.stages; ++s) mbar_init(reinterpret_cast<uint64_t*>(dsm) + s, 1);
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
        if (alive) {
            alive = mbar_wait(&bar[st], phase, pl.fault);
            if (!alive) failed_at = k;
        }
        if (!body(b, dsm + 128 + (size_t)st * pl.stage_bytes, alive)) __syncthreads();
        if (threadIdx.x < 32 && alive && k + pl.stages < K) {
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

// The bytes of vector `gb` (its byte offset in a contiguous input) that the
// ring did not copy, one element of E bytes at a time; elements outside the
// mask are zeros.
template <int E, int VEC, int NW>
__device__ __forceinline__ void gather_tail(const RowSrc& s, int64_t gb, uint32_t em,
                                            uint32_t (&v)[NW])
{
#pragma unroll
    for (int i = 0; i < NW; ++i) v[i] = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
        if ((em >> e) & 1u) {
            const unsigned char* p = s.p + gb + e * E;
            if constexpr (E == 1)
                v[e / 4] |= (uint32_t)*p << (8 * (e % 4));
            else if constexpr (E == 2)
                v[e / 2] |= (uint32_t)*reinterpret_cast<const unsigned short*>(p) << (16 * (e % 2));
            else
                v[e] = *reinterpret_cast<const uint32_t*>(p);
        }
}

// Words of the elements in the mask, zeros for the others.
template <int VEC, int NW>
__device__ __forceinline__ void mask_words(uint32_t (&v)[NW], uint32_t em)
{
    constexpr int per = VEC / NW;  // elements a word
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < per; ++e)
            if ((em >> (i * per + e)) & 1u) m |= (per == 1 ? ~0u : ((1u << (32 / per)) - 1u)) << (e * (32 / per) % 32);
        v[i] &= m;
    }
}

// Vector at byte `off` of the slot (16 bytes of activations).  `last`: the
// block may reach past the copied bytes; gb is then its byte offset in the
// input.
template <typename TX, bool kEdge>
__device__ __forceinline__ uint4 ld_vec(const unsigned char* slot, uint32_t off, bool ok,
                                        const RowSrc& s, bool last, int64_t gb, uint32_t em)
{
    if constexpr (kEdge) {
        uint32_t v[4] = {0, 0, 0, 0};
        if (ok) {
            if (last && gb + 16 > (s.total & ~(int64_t)15)) {
                gather_tail<sizeof(TX), Vec<TX>::kN>(s, gb, em, v);
            } else {
                const uint4 q = lds128(slot + off);
                v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
                if (em != (1u << Vec<TX>::kN) - 1u) mask_words<Vec<TX>::kN>(v, em);
            }
        }
        return make_uint4(v[0], v[1], v[2], v[3]);
    } else {
        return lds128_if(ok, slot + off);
    }
}

// A vector's VEC 8-bit values, from the slot (or past the copied bytes).
template <int VEC, bool kEdge>
__device__ __forceinline__ void ld_vec8(uint32_t (&v)[VEC / 4], const unsigned char* slot,
                                        uint32_t off, bool ok, const RowSrc& s, bool last,
                                        int64_t gb, uint32_t em)
{
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) v[i] = 0;
    if (!ok) return;
    if (last && gb + VEC > (s.total & ~(int64_t)15)) {
        gather_tail<1, VEC>(s, gb, em, v);
        return;
    }
    if constexpr (VEC == 8) {
        const uint2 q = lds64(slot + off);
        v[0] = q.x;
        v[1] = q.y;
    } else {
        v[0] = lds32(slot + off);
    }
    if constexpr (kEdge)
        if (em != (1u << VEC) - 1u) mask_words<VEC>(v, em);
}

// Store a vector of activations: whole, or the elements in the mask.
template <typename TX, bool kEdge>
__device__ __forceinline__ void st_vec(TX* p, const uint4& v, bool ok, uint32_t em)
{
    if constexpr (kEdge) {
        if (!ok) return;
        if (em == (1u << Vec<TX>::kN) - 1u) {
            st_stream(p, v);
            return;
        }
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
    } else {
        st_stream_if(ok, p, v);
    }
}

template <int VEC, bool kEdge>
__device__ __forceinline__ void st_vec8(unsigned char* p, const uint32_t (&v)[VEC / 4], bool ok,
                                        uint32_t em)
{
    if (!ok) return;
    if (kEdge && em != (1u << VEC) - 1u) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if ((em >> e) & 1u) p[e] = (unsigned char)(v[e / 4] >> (8 * (e % 4)));
        return;
    }
    if constexpr (VEC == 8)
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(v[0], v[1]));
    else
        __stcs(reinterpret_cast<unsigned*>(p), v[0]);
}

// A thread's part of its rows: its vector j is vector l + j W of the row,
// whose element 0 is column col(j) = (l + j W) VEC - first, and em[j] says
// which of its elements are the row's.
template <int VEC, int KV, bool kEdge>
struct Cols {
    int l, W, first;
    uint32_t em[KV];
    __device__ Cols(int lane, int W_, int first_, int N)
        : l(lane), W(W_), first(kEdge ? first_ : 0)
    {
#pragma unroll
        for (int j = 0; j < KV; ++j) {
            const int c = col(j), lo = c < 0 ? -c : 0, hi = N - c < VEC ? N - c : VEC;
            em[j] = hi > lo ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
        }
    }
    __device__ int vec(int j) const { return l + j * W; }
    __device__ int col(int j) const { return vec(j) * VEC - first; }
    __device__ bool ok(int j) const { return em[j] != 0; }
};

// Weights of a thread's vectors as float32 (1 + w for Gemma), zeros outside
// the row.  Whole vectors of an aligned weight come as 16-byte loads.
template <int VEC, int KV, bool kEdge>
__device__ __forceinline__ void load_weights(f2 (&wf)[KV][VEC / 2], const Cols<VEC, KV, kEdge>& c,
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
                    const float4 v =
                        __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + c.col(j)) + q);
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

// Sums (and NaN-keeping maxima) over a row group, U rows at once: every
// thread of a group gets the same bits.  kW > 0: a group is kW <= 32 lanes of
// a warp.  kW 0: a group of up to kWarps whole warps, joined through `red`
// (row_red_floats, zero where no warp writes) with one __syncthreads; the two
// halves of red are used in turn.
template <int kW, int kWarps, int G, int U, bool kMax>
__device__ __forceinline__ void row_reduce(float (&s)[U], float (&m)[U], float* red, int& parity,
                                           int g, int l)
{
    constexpr int kIn = kW ? kW : 32;
    butterfly<kIn, U>(s);
    if constexpr (kMax) {
#pragma unroll
        for (int off = kIn / 2; off >= 1; off >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u)
                m[u] = max_nan(m[u], __shfl_xor_sync(0xffffffffu, m[u], off));
    }
    if constexpr (kW == 0) {
        constexpr int kV = kMax ? 2 * U : U;
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
template <int kW, int kWarps, int G, int U, bool kMax>
constexpr int row_red_floats()
{
    return kW ? 1 : 2 * G * (kMax ? 2 * U : U) * kWarps;
}
// Zero red; the caller's next __syncthreads publishes it.
template <int kFloats>
__device__ __forceinline__ void row_red_init(float* red)
{
    for (int i = threadIdx.x; i < kFloats; i += blockDim.x) red[i] = 0.f;
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
        default: return false;
    }
}

#endif  // __CUDACC__

}  // namespace gbn
