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

// Row groups: rows of up to `cap` vectors go to W threads with KV vectors
// each, of CTAs of T threads.  One vector a thread up to a warp's 32, then
// two: half the warps, and half the reduction, that one would take.
struct RowSched {
    int cap, W, T, KV;
};
constexpr int kNumRowSched = 10;
constexpr RowSched kRow[kNumRowSched] = {
    {4, 4, 256, 1},    {8, 8, 256, 1},     {16, 16, 256, 1},   {32, 32, 256, 1},
    {64, 32, 256, 2},  {128, 64, 256, 2},  {256, 128, 256, 2}, {512, 256, 256, 2},
    {1024, 512, 512, 2}, {2048, 1024, 1024, 2},
};
// Rows a thread takes of a block, CTAs an SM, ring stages.
constexpr int row_U(int S) { return kRow[S].KV == 1 ? 2 : 1; }
constexpr int row_R(int S) { return kRow[S].T / kRow[S].W * row_U(S); }
constexpr int fwd_minb(int S, bool edge)
{
    return kRow[S].T == 256 ? (kRow[S].KV == 1 && !edge ? 4 : 3)
           : kRow[S].T == 512 && !edge ? 2 : 1;
}
constexpr int bwd_minb(int S) { return kRow[S].T == 256 ? 2 : 1; }
constexpr int fwd_stages(int S) { return kRow[S].T == 256 ? 2 : 3; }
// Dynamic shared memory the kernels may ask for: three inputs of the widest
// rows (32 KB each) in two stages, and room for the group maxima.
constexpr int kMaxSmem = 208 * 1024;
constexpr int bwd_stages(int S) { return kRow[S].T == 1024 ? 2 : 3; }

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
// Byte offset in the slot of row i (of the block from row r0 on): its first
// vector, on a 16-byte boundary for the storage's vectors of 16 bytes.
__device__ __forceinline__ uint32_t row_off(const RowSrc& s, int64_t r0, int i)
{
    const uint32_t rb = (uint32_t)s.row_bytes;
    return (s.scattered ? 0u : (uint32_t)(r0 * s.row_bytes) & 15u) + (uint32_t)i * rb;
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

// A thread's part of its rows: element 0 of its vector j is column
// col(j) = (l + j W) VEC - first, and em[j] says which of its elements are
// the row's.
template <int VEC, int W, int KV, bool kEdge>
struct Cols {
    int l, first;
    uint32_t em[KV];
    __device__ Cols(int lane, int first_, int N) : l(lane), first(kEdge ? first_ : 0)
    {
#pragma unroll
        for (int j = 0; j < KV; ++j) {
            const int c = col(j), lo = c < 0 ? -c : 0, hi = N - c < VEC ? N - c : VEC;
            em[j] = hi > lo ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
        }
    }
    __device__ int col(int j) const { return (l + j * W) * VEC - first; }
    __device__ bool ok(int j) const { return em[j] != 0; }
};

// Weights of a thread's vectors as float32 (1 + w for Gemma), zeros outside
// the row.
template <int VEC, int W, int KV, bool kEdge>
__device__ __forceinline__ void load_weights(f2 (&wf)[KV][VEC / 2], const Cols<VEC, W, KV, kEdge>& c,
                                             const void* w, int wt, bool gemma)
{
#pragma unroll
    for (int j = 0; j < KV; ++j)
#pragma unroll
        for (int p = 0; p < VEC / 2; ++p) {
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = (c.em[j] >> (2 * p + h)) & 1u;
                v[h] = in ? ld_param(w, wt, c.col(j) + 2 * p + h) + (gemma ? 1.f : 0.f) : 0.f;
            }
            wf[j][p] = mk2(v[0], v[1]);
        }
}

// Sums (and NaN-keeping maxima) over the W threads of a row group, U rows at
// once: every thread of a group gets the same bits.  Groups of several warps
// join through `red` (2 x (T / W) x 2U x 32 floats, used in turn) with one
// __syncthreads.
template <int W, int T, int U, bool kMax>
__device__ __forceinline__ void row_reduce(float (&s)[U], float (&m)[U], float* red, int& parity)
{
    constexpr int kIn = W < 32 ? W : 32;
    butterfly<kIn, U>(s);
    if constexpr (kMax)
#pragma unroll
        for (int off = kIn / 2; off >= 1; off >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u)
                m[u] = max_nan(m[u], __shfl_xor_sync(0xffffffffu, m[u], off));
    if constexpr (W > 32) {
        constexpr int kWarps = W / 32, kG = T / W, kV = kMax ? 2 * U : U;
        const int lane = threadIdx.x & 31, g = threadIdx.x / W, wig = (threadIdx.x % W) >> 5;
        float* slot = red + (parity * kG + g) * kV * 32;
        if (lane == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                slot[u * 32 + wig] = s[u];
                if constexpr (kMax) slot[(U + u) * 32 + wig] = m[u];
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = slot[u * 32 + (lane & (kWarps - 1))];
            if constexpr (kMax) m[u] = slot[(U + u) * 32 + (lane & (kWarps - 1))];
        }
        butterfly<kWarps, U>(s);
        if constexpr (kMax)
#pragma unroll
            for (int off = kWarps / 2; off >= 1; off >>= 1)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    m[u] = max_nan(m[u], __shfl_xor_sync(0xffffffffu, m[u], off));
        parity ^= 1;
    }
}
template <int W, int T, int U, bool kMax>
constexpr int row_red_floats()
{
    return W > 32 ? 2 * (T / W) * (kMax ? 2 * U : U) * 32 : 1;
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
