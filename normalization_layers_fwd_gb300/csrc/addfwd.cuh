// addfwd.cuh -- the ring kernel of the residual-stream forwards: s = x + res,
// its RMSNorm in x's type or in 8 bits, the 8-bit checkpoint of s, and (mode
// kModeC) the checkpoint alone.  addfwd_*.cu instantiate it.
//
// One pass: a thread adds and rounds its vectors of s and keeps them, packed,
// over the row reduction; the maxima for the 8-bit scales go with it (the
// output's largest magnitude is r times that of w s, so it needs no second
// walk).  Everything read is read once and everything written once, so HBM
// bounds it.  Measured (bf16, of measured copy bandwidth, graph of passes):
// y [65536, 1024] 84 us, 0.94; y [16384, 4096] 88 us, 0.90; 8-bit output
// [16384, 4096] 76 us, 0.92; y with its checkpoint 100 us, 0.89.
// Rows that start inside a vector (odd N) pay for their masked ends and, with
// groups, for maxima that meet in shared memory: y N = 3001 0.90, 8-bit output
// 0.47, where the warps' instructions bound it.
#pragma once

#include "rowring.cuh"

namespace gbn {
namespace {

// VEC values times k as 8-bit codes.
template <int VEC, int kType>
__device__ __forceinline__ void pack_vec8(uint32_t (&out)[VEC / 4], const f2 (&v)[VEC / 2], float k)
{
    const f2 kk = splat2(k);
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) out[i] = q8_pack4<kType>(v[2 * i], v[2 * i + 1], kk, kk);
}

// Bytes (of VEC / 4 words) or 16-bit halves (of VEC / 2) of the elements
// before eb.
template <int VEC, int NW>
__device__ __forceinline__ void before(uint32_t (&m)[NW], int eb)
{
#pragma unroll
    for (int i = 0; i < NW; ++i) m[i] = ~0u;
    mask_words<VEC>(m, (1u << eb) - 1u);
}

template <typename TX, int S, bool kEdge, int kFull>
__global__ void __launch_bounds__(row_sched(fwd_kind(kFull), S).T, row_minb(fwd_kind(kFull), S))
    add_fwd_ring(const __grid_constant__ FwdArgs a, const __grid_constant__ RowPlan pl)
{
    grid_dependency_sync();
    constexpr int kMode = kFull & 3, kType = kFull >= kModeInt8 ? kInt8 : kE4M3;
    constexpr int kKind = fwd_kind(kMode), kW = row_sched(kKind, S).W, KV = row_sched(kKind, S).KV;
    constexpr int U = row_U(kKind, S), kG = row_G(kKind, S), kLanes = kW ? kW : 256;
    constexpr int VEC = Vec<TX>::kN, P = VEC / 2, E = (int)sizeof(TX);
    constexpr bool kNorm = kMode != kModeC, kMax = kMode != kModeY;
    constexpr int kRed = row_red_floats<kLanes, kG, U, kMax>();
    extern __shared__ __align__(128) unsigned char dsm[];
    __shared__ float red[kRed];
    int parity = 0;
    const int N = a.N, W = kW ? kW : pl.W, G = kW ? kG : pl.G, R = G * U;
    const int g = threadIdx.x / W, l = threadIdx.x - g * W;
    if constexpr (kW == 0)
        for (int i = threadIdx.x; i < kRed; i += W * G) red[i] = 0.f;
    const int64_t K = row_ring_start(a.in, pl, a.M, dsm);

    // the first row of this thread; its later ones are a multiple of VEC rows on
    int64_t row = (int64_t)blockIdx.x * R + g;
    const Cols<VEC, kW, KV, kEdge> cols(l, W, kEdge ? (int)(row * N % VEC) : 0, N);
    f2 wf[KV][P];
    if constexpr (kNorm) load_weights<VEC, kW, KV, kEdge>(wf, cols, a.w, a.wt, a.variant == 2);
    // this thread's first vector: its element in the [M, N] tensors, and its
    // byte in a slot (rows of a slot are row_bytes apart)
    int64_t at = row * N - cols.first + l * VEC;
    const int64_t row_step = (int64_t)gridDim.x * R, at_step = row_step * N;
    const uint32_t so0 = pl.off[0] + row_off(a.in[0], row - g, g) - cols.first * E + l * 16;
    const uint32_t so1 = pl.off[1] + row_off(a.in[1], row - g, g) - cols.first * E + l * 16;
    const uint32_t srow = (uint32_t)G * (uint32_t)a.in[0].row_bytes;

    // 8-bit groups: the output's or the checkpoint's
    const Q8& q8 = kMode == kModeQ ? a.q : a.c;
    const bool whole = q8.shift == 31;              // a scale per row
    const int lanes = whole ? W : (1 << q8.shift) / VEC;  // of a group, when rows are whole vectors
    // Groups of rows that start inside a vector (kEdge): a vector's elements
    // before eb belong to group ga, the others to the next one.  (W VEC is a
    // multiple of a group, so eb is the same for all of a thread's vectors;
    // the row's first vector, which starts before it, has ga = -1.)  Their
    // maxima meet in shared memory: gm[2][R][ng], used in turn.
    const bool cutg = kEdge && kMax && !whole;
    constexpr int kIn = kLanes < 32 ? kLanes : 32;
    const int shift = kEdge && cols.first != 0 ? 1 : 0;  // lanes by which runs of a group are off
    int ga0 = 0, eb = VEC;
    if (kMax && !whole) {
        ga0 = cols.col(0) >> q8.shift;
        if (kEdge) {
            eb = ((ga0 + 1) << q8.shift) - cols.col(0);
            eb = eb < VEC ? eb : VEC;
        }
    }
    const int gstep = whole ? 0 : (W * VEC) >> q8.shift;
    uint32_t m16[VEC / 2], m8[VEC / 4];
    before<VEC, VEC / 2>(m16, eb);
    before<VEC, VEC / 4>(m8, eb);
    unsigned* const gm = reinterpret_cast<unsigned*>(dsm + pl.gm_off);
    float* const rsm = reinterpret_cast<float*>(gm + 2 * R * q8.ng);
    if (cutg) {
        for (int i = threadIdx.x; i < 2 * R * q8.ng; i += W * G) gm[i] = 0;
        __syncthreads();
    }
    int half = 0;  // of gm

    row_ring(a.in, pl, a.M, dsm, K, [&](int64_t b, const unsigned char* slot, bool alive) {
        const bool last = b == pl.nblocks - 1;
        uint4 sp[U][KV];
        float ss[U], mx[U], gmx[U][KV];
        bool okr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            okr[u] = alive && (!last || row + u * G < a.M);
            ss[u] = 0.f;
            mx[u] = 0.f;
            TX* const sr = static_cast<TX*>(a.s) + at + (int64_t)u * G * N;
#pragma unroll
            for (int j = 0; j < KV; ++j) {
                gmx[u][j] = 0.f;
                sp[u][j] = make_uint4(0, 0, 0, 0);
                if (KV > 1 && j >= cols.live) continue;
                const bool ok = okr[u] && cols.ok(j);
                const uint32_t o = u * srow + j * W * 16;
                sp[u][j] = ld_vec<TX>(slot, so0 + o, ok, cols.cut(j), cols.em[j]);
                if (a.in[1].p) {
                    const uint4 rv =
                        ld_vec<TX>(slot, so1 + o, ok, cols.cut(j), cols.em[j]);
                    f2 xa[P], xb[P];
                    unpack2<TX>(sp[u][j], xa);
                    unpack2<TX>(rv, xb);
#pragma unroll
                    for (int p = 0; p < P; ++p) xa[p] = add2(xa[p], xb[p]);
                    sp[u][j] = pack2<TX>(xa);  // the stream, rounded once
                    if (a.s)
                        st_vec<TX>(sr + j * W * VEC, sp[u][j], ok, cols.cut(j), cols.em[j]);
                }
                f2 sv[P];
                unpack2<TX>(sp[u][j], sv);
                if constexpr (kNorm) {
                    f2 q = splat2(0.f);
#pragma unroll
                    for (int p = 0; p < P; ++p) q = fma2(sv[p], sv[p], q);
                    ss[u] += lo2(q) + hi2(q);
                }
                if constexpr (kMax) {
                    if constexpr (kMode == kModeQ) {
#pragma unroll
                        for (int p = 0; p < P; ++p) sv[p] = mul2(sv[p], wf[j][p]);
                    }
                    auto amax = [&](const f2 (&v)[P]) {
                        float m = 0.f;
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            m = max_nan(max_nan(m, fabsf(lo2(v[p]))), fabsf(hi2(v[p])));
                        return m;
                    };
                    if (!cutg) {
                        const float m = kMode == kModeQ ? amax(sv) : vec_amax<TX>(sp[u][j]);
                        gmx[u][j] = m;
                        mx[u] = max_nan(mx[u], m);
                    } else {
                        // both groups' shares; the second goes to the next lane,
                        // whose vector starts in that group
                        const int ga = ga0 + j * gstep;
                        float ma, mb;
                        if constexpr (kMode != kModeQ && is16<TX>()) {
                            const uint4 v = sp[u][j];
                            ma = vec_amax<TX>(make_uint4(v.x & m16[0], v.y & m16[1], v.z & m16[2],
                                                         v.w & m16[3]));
                            mb = vec_amax<TX>(make_uint4(v.x & ~m16[0], v.y & ~m16[1],
                                                         v.z & ~m16[2], v.w & ~m16[3]));
                        } else {
                            f2 va[P], vb[P];
#pragma unroll
                            for (int p = 0; p < P; ++p) {
                                const bool b0 = 2 * p < eb, b1 = 2 * p + 1 < eb;
                                va[p] = mk2(b0 ? lo2(sv[p]) : 0.f, b1 ? hi2(sv[p]) : 0.f);
                                vb[p] = mk2(b0 ? 0.f : lo2(sv[p]), b1 ? 0.f : hi2(sv[p]));
                            }
                            ma = amax(va);
                            mb = amax(vb);
                        }
                        const bool two = ok && eb < VEC && ga + 1 < q8.ng;
                        const float up = __shfl_up_sync(0xffffffffu, two ? mb : 0.f, 1, kIn);
                        const int lane = l & (kIn - 1);
                        if (lane != 0) ma = max_nan(ma, up);
                        // The lanes of a warp that share a group: aligned runs of
                        // `lanes`, one lane further on where rows start inside a
                        // vector (lane 0 then ends a run of the warp before and
                        // stays out).  Magnitudes compare like their bits (NaN on
                        // top): one atomic a run, whose order does not matter.
                        const bool out = shift && lane == 0;
                        float m = out ? 0.f : ma;
                        const int place = (lane - shift) & (kIn - 1);
                        for (int off = 1; off < lanes; off <<= 1) {
                            const int from = ((place ^ off) + shift) & (kIn - 1);
                            m = max_nan(m, __shfl_sync(0xffffffffu, m, from, kIn));
                        }
                        unsigned* const dst = gm + (half * R + g + u * G) * q8.ng + ga;
                        if (ok && ga >= 0 && (out || ((lane - shift) & (lanes - 1)) == 0))
                            atomicMax(dst, __float_as_uint(out ? ma : m));
                        if (two && (lane == kIn - 1 || cols.col(j) + VEC >= N))  // no next lane
                            atomicMax(dst + 1, __float_as_uint(mb));
                    }
                }
            }
        }
        // the row's sum, and its maximum for a scale per row; a group's
        // maximum from its lanes, or from shared memory
        if (kNorm || whole) row_reduce<kLanes, kG, U, kMax>(ss, mx, red, parity, g, l);
        float rs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) rs[u] = kNorm ? rsqrtf(fmaf(ss[u], a.inv_n, a.eps)) : 1.f;
        if (cutg) {
            // a thread per group: its scale, and the factor its elements take
            if (l == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) rsm[g + u * G] = kMode == kModeQ ? rs[u] : 1.f;
            }
            __syncthreads();
            unsigned* const now = gm + half * R * q8.ng;
            half ^= 1;
            unsigned* const next = gm + half * R * q8.ng;
            for (int i = threadIdx.x; i < R * q8.ng; i += W * G) {
                const int q = i / q8.ng;  // the row
                const float t = rsm[q], sc = q8_scale(__uint_as_float(now[i]) * t, kType);
                now[i] = __float_as_uint(t * __frcp_rn(sc));
                next[i] = 0;
                if (alive && b * R + q < a.M) q8.scale[b * R * q8.ng + i] = sc;
            }
            __syncthreads();
        } else if (kMax && !whole) {
            for (int off = 1; off < lanes; off <<= 1)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < KV; ++j)
                        gmx[u][j] =
                            max_nan(gmx[u][j], __shfl_xor_sync(0xffffffffu, gmx[u][j], off));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = row + u * G;
            const f2 r2 = splat2(rs[u]);
            if (kNorm && a.rstd) st_f32_if(l == 0 && okr[u], a.rstd + r, rs[u]);
            const int64_t atu = at + (int64_t)u * G * N;
#pragma unroll
            for (int j = 0; j < KV; ++j) {
                if (KV > 1 && j >= cols.live) continue;
                const bool ok = okr[u] && cols.ok(j);
                f2 sv[P];
                unpack2<TX>(sp[u][j], sv);
                if constexpr (kMode == kModeY || kMode == kModeYC) {
                    uint4 o;
                    f2 f[P];
                    if constexpr (is16<TX>()) {
                        if (a.variant != 0) {
#pragma unroll
                            for (int p = 0; p < P; ++p) f[p] = mul2(wf[j][p], mul2(sv[p], r2));
                            o = pack2<TX>(f);
                        } else if (a.wt == dtype_code<TX>()) {
                            // n = rx(s r), y = rx(w n): a product of 16-bit values, rounded once
                            uint32_t h[4];
#pragma unroll
                            for (int p = 0; p < P; ++p)
                                h[p] = P16<TX>::mul(P16<TX>::from_f2(wf[j][p]),
                                                    P16<TX>::from_f2(mul2(sv[p], r2)));
                            o = make_uint4(h[0], h[1], h[2], h[3]);
                        } else {
#pragma unroll
                            for (int p = 0; p < P; ++p)
                                f[p] = mul2(wf[j][p], round2<TX>(mul2(sv[p], r2)));
                            o = pack2<TX>(f);
                        }
                    } else {
#pragma unroll
                        for (int p = 0; p < P; ++p) f[p] = mul2(wf[j][p], mul2(sv[p], r2));
                        o = pack2<TX>(f);
                    }
                    st_vec<TX>(static_cast<TX*>(a.y) + atu + j * W * VEC, o, ok,
                               cols.cut(j), cols.em[j]);
                }
                if constexpr (kMax) {
                    if constexpr (kMode == kModeQ) {
#pragma unroll
                        for (int p = 0; p < P; ++p) sv[p] = mul2(sv[p], wf[j][p]);
                    }
                    uint32_t o[VEC / 4];
                    const int ga = ga0 + j * gstep;
                    if (cutg) {
                        // the other half of gm: `half` was turned
                        const unsigned* k = gm + ((half ^ 1) * R + g + u * G) * q8.ng + ga;
                        const bool two = ok && eb < VEC && ga + 1 < q8.ng;
                        const float ka = ok && ga >= 0 ? __uint_as_float(k[0]) : 0.f;
                        const float kb = two ? __uint_as_float(k[1]) : 0.f;
                        uint32_t ob[VEC / 4];
                        pack_vec8<VEC, kType>(o, sv, ka);
                        pack_vec8<VEC, kType>(ob, sv, kb);
#pragma unroll
                        for (int i = 0; i < VEC / 4; ++i) o[i] = (o[i] & m8[i]) | (ob[i] & ~m8[i]);
                    } else {
                        const float t = kMode == kModeQ ? rs[u] : 1.f;  // r enters here
                        const float sc = q8_scale((whole ? mx[u] : gmx[u][j]) * t, kType);
                        pack_vec8<VEC, kType>(o, sv, t * __frcp_rn(sc));
                        // the vector that holds a group's first column writes its scale
                        const int c = cols.col(j) < 0 ? 0 : cols.col(j);
                        if (ok && (c & (whole ? -1 : (1 << q8.shift) - 1)) == 0)
                            q8.scale[r * q8.ng + ga] = sc;
                    }
                    st_vec8<VEC>(static_cast<unsigned char*>(q8.v) + atu + j * W * VEC, o, ok,
                                 cols.cut(j), cols.em[j]);
                }
            }
        }
        row += row_step;
        at += at_step;
        // a barrier came after the last read of the slot
        return cutg || (kLanes > 32 && (kNorm || whole));
    });
}

template <typename TX>
cudaError_t fwd_launch(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p)
{
    auto go = [&](auto s_, auto edge_, auto mode_) {
        constexpr int S = decltype(s_)::value, kMode = decltype(mode_)::value;
        constexpr bool kEdge = decltype(edge_)::value;
        if constexpr (row_takes(fwd_kind(kMode), S)) {
            ring_attributes<add_fwd_ring<TX, S, kEdge, kMode>>(kMaxSmem);
            launch_pdl(add_fwd_ring<TX, S, kEdge, kMode>, p.grid, p.W * p.G, p.smem, st, a, p);
        }
    };
    auto modes = [&](auto s_, auto edge_) {
        using std::integral_constant;
        switch (mode) {
            case kModeY: go(s_, edge_, integral_constant<int, kModeY>{}); break;
            case kModeQ: go(s_, edge_, integral_constant<int, kModeQ>{}); break;
            case kModeYC: go(s_, edge_, integral_constant<int, kModeYC>{}); break;
            case kModeQ + kModeInt8:
                go(s_, edge_, integral_constant<int, kModeQ + kModeInt8>{});
                break;
            case kModeYC + kModeInt8:
                go(s_, edge_, integral_constant<int, kModeYC + kModeInt8>{});
                break;
            case kModeC + kModeInt8:
                go(s_, edge_, integral_constant<int, kModeC + kModeInt8>{});
                break;
            default: go(s_, edge_, integral_constant<int, kModeC>{}); break;
        }
    };
    const bool found = with_row_sched(p.sid, [&](auto s_) {
        if (p.edge)
            modes(s_, std::true_type{});
        else
            modes(s_, std::false_type{});
    });
    return found ? cudaGetLastError() : cudaErrorInvalidValue;
}

}  // namespace
}  // namespace gbn
