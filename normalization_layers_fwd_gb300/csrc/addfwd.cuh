// addfwd.cuh -- the ring kernel of the residual-stream forwards: s = x + res,
// its RMSNorm in x's type or in 8 bits, the 8-bit checkpoint of s, and (mode
// kModeC) the checkpoint alone.  One pass: a thread adds and rounds its
// vectors of s and keeps them, packed, over the row reduction; the maxima for
// the 8-bit scales go with it (the output's largest magnitude is r times
// that of w s, so it needs no second walk).  addfwd_*.cu instantiate it.
#pragma once

#include "rowring.cuh"

namespace gbn {
namespace {

// VEC values times k (ka before element eb, kb from it on) as 8-bit codes.
template <int VEC, bool kTwo, int kType>
__device__ __forceinline__ void pack_vec8(uint32_t (&out)[VEC / 4], const f2 (&v)[VEC / 2],
                                          float ka, float kb, int eb)
{
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        f2 k0 = splat2(ka), k1 = k0;
        if constexpr (kTwo) {
            k0 = mk2(4 * i < eb ? ka : kb, 4 * i + 1 < eb ? ka : kb);
            k1 = mk2(4 * i + 2 < eb ? ka : kb, 4 * i + 3 < eb ? ka : kb);
        }
        out[i] = q8_pack4<kType>(v[2 * i], v[2 * i + 1], k0, k1);
    }
}

template <typename TX, int S, bool kEdge, int kFull>
__global__ void __launch_bounds__(row_sched(fwd_kind(kFull), S).T, row_minb(fwd_kind(kFull), S, kEdge))
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
    // kEdge: a vector's elements before eb belong to group ga, the others to the next
    int ga[KV], eb[KV];
    bool lead[KV];  // the vector holds its group's first column
    constexpr int kIn = kLanes < 32 ? kLanes : 32;
    const int shift = kEdge && cols.first != 0 ? 1 : 0;
    float* const gm = reinterpret_cast<float*>(dsm + pl.gm_off);  // [2][R][ng] maxima (kEdge)
    const bool shared_max = kEdge && kMax && !whole;
    if constexpr (kMax) {
#pragma unroll
        for (int j = 0; j < KV; ++j) {
            const int c = cols.col(j) < 0 ? 0 : cols.col(j);
            ga[j] = whole ? 0 : c >> q8.shift;
            eb[j] = kEdge && !whole ? ((ga[j] + 1) << q8.shift) - cols.col(j) : VEC;
            lead[j] = cols.ok(j) && (c & (whole ? -1 : (1 << q8.shift) - 1)) == 0;
        }
        if (shared_max) {
            for (int i = threadIdx.x; i < 2 * R * q8.ng; i += W * G) gm[i] = 0.f;
            __syncthreads();
        }
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
                    if (!shared_max) {
                        float m = 0.f;
                        if constexpr (kMode == kModeQ) {
#pragma unroll
                            for (int p = 0; p < P; ++p)
                                m = max_nan(max_nan(m, fabsf(lo2(sv[p]))), fabsf(hi2(sv[p])));
                        } else {
                            m = vec_amax<TX>(sp[u][j]);
                        }
                        gmx[u][j] = m;
                        mx[u] = max_nan(mx[u], m);
                    } else {
                        // both groups' shares; the second goes to the next lane,
                        // whose vector starts in that group
                        float ma = 0.f, mb = 0.f;
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            const float lo = fabsf(lo2(sv[p])), hi = fabsf(hi2(sv[p]));
                            if (2 * p < eb[j]) ma = max_nan(ma, lo); else mb = max_nan(mb, lo);
                            if (2 * p + 1 < eb[j]) ma = max_nan(ma, hi); else mb = max_nan(mb, hi);
                        }
                        const bool two = ok && eb[j] < VEC && ga[j] + 1 < q8.ng;
                        const float up = __shfl_up_sync(0xffffffffu, two ? mb : 0.f, 1, kIn);
                        if ((l & (kIn - 1)) != 0) ma = max_nan(ma, up);
                        // the lanes of a warp that share a group: aligned runs of
                        // `lanes`, one lane further on where rows start inside a
                        // vector (lane 0 then ends a run of the warp before and
                        // stays out).  Magnitudes compare like their bits (NaN on
                        // top): one atomic a run, whose order does not matter
                        const bool out = shift && (l & (kIn - 1)) == 0;
                        float m = out ? 0.f : ma;
                        for (int off = 1; off < lanes; off <<= 1)
                            m = max_nan(m, __shfl_sync(0xffffffffu, m,
                                                       ((((l - shift) & (kIn - 1)) ^ off) + shift) & (kIn - 1), kIn));
                        unsigned* const dst = reinterpret_cast<unsigned*>(gm) +
                                              (half * R + g + u * G) * q8.ng + ga[j];
                        if (ok && (out || ((l - shift) & (lanes - 1)) == 0))
                            atomicMax(dst, __float_as_uint(out ? ma : m));
                        if (two && ((l & (kIn - 1)) == kIn - 1 ||
                                    cols.col(j) + VEC >= N))  // no next lane to take it
                            atomicMax(dst + 1, __float_as_uint(mb));
                    }
                }
            }
        }
        // the row's sum, and its maximum for a scale per row; a group's
        // maximum from its lanes, or from shared memory
        if (kNorm || whole) row_reduce<kLanes, kG, U, kMax>(ss, mx, red, parity, g, l);
        if constexpr (kMax) {
            if (shared_max) {
                __syncthreads();
            } else if (!whole) {
                for (int off = 1; off < lanes; off <<= 1)
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int j = 0; j < KV; ++j)
                            gmx[u][j] = max_nan(gmx[u][j],
                                                __shfl_xor_sync(0xffffffffu, gmx[u][j], off));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = row + u * G;
            const float rs = kNorm ? rsqrtf(fmaf(ss[u], a.inv_n, a.eps)) : 1.f;
            const f2 r2 = splat2(rs);
            if (kNorm && a.rstd) st_f32_if(l == 0 && okr[u], a.rstd + r, rs);
            const int64_t atu = at + (int64_t)u * G * N;
#pragma unroll
            for (int j = 0; j < KV; ++j) {
                if (KV > 1 && j >= cols.live) continue;
                const bool ok = okr[u] && cols.ok(j);
                f2 sv[P];
                unpack2<TX>(sp[u][j], sv);
                if constexpr (kMode == kModeY || kMode == kModeYC) {
                    f2 o[P];
                    if (is16<TX>() && a.variant == 0) {
#pragma unroll
                        for (int p = 0; p < P; ++p)  // n = rx(s r), y = rx(w n)
                            o[p] = mul2(wf[j][p], round2<TX>(mul2(sv[p], r2)));
                    } else {
#pragma unroll
                        for (int p = 0; p < P; ++p) o[p] = mul2(wf[j][p], mul2(sv[p], r2));
                    }
                    st_vec<TX>(static_cast<TX*>(a.y) + atu + j * W * VEC, pack2<TX>(o), ok,
                               cols.cut(j), cols.em[j]);
                }
                if constexpr (kMax) {
                    float ma = whole ? mx[u] : gmx[u][j], mb = 0.f;
                    if (shared_max && ok) {
                        const float* m = gm + (half * R + g + u * G) * q8.ng + ga[j];
                        ma = m[0];
                        mb = eb[j] < VEC && ga[j] + 1 < q8.ng ? m[1] : 0.f;
                    }
                    if constexpr (kMode == kModeQ) {
#pragma unroll
                        for (int p = 0; p < P; ++p) sv[p] = mul2(sv[p], wf[j][p]);
                    }
                    const float t = kMode == kModeQ ? rs : 1.f;  // r enters here
                    const float sa = q8_scale(ma * t, kType);
                    const float ka = t * __frcp_rn(sa);
                    float sb = 0.f, kb = ka;
                    if (shared_max) {
                        sb = q8_scale(mb * t, kType);
                        kb = t * __frcp_rn(sb);
                    }
                    uint32_t o[VEC / 4];
                    pack_vec8<VEC, kEdge, kType>(o, sv, ka, kb, eb[j]);
                    st_vec8<VEC>(static_cast<unsigned char*>(q8.v) + atu + j * W * VEC, o, ok,
                                 cols.cut(j), cols.em[j]);
                    // the vector that holds a group's first column writes its scale
                    float* const sc = q8.scale + r * q8.ng + ga[j];
                    if (okr[u] && lead[j]) sc[0] = sa;
                    if (shared_max && ok && eb[j] < VEC && ga[j] + 1 < q8.ng) sc[1] = sb;
                }
            }
        }
        row += row_step;
        at += at_step;
        if (shared_max) {
            // the other half is free: its readers passed the barrier above
            half ^= 1;
            for (int i = threadIdx.x; i < R * q8.ng; i += W * G) gm[half * R * q8.ng + i] = 0.f;
            return false;  // and a barrier before its next use
        }
        return kLanes > 32 && (kNorm || whole);  // row_reduce's barrier came after the last slot read
    });
}

template <typename TX>
cudaError_t fwd_launch(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p)
{
    auto go = [&](auto s_, auto edge_, auto mode_) {
        constexpr int S = decltype(s_)::value, kMode = decltype(mode_)::value;
        constexpr bool kEdge = decltype(edge_)::value;
        ring_attributes<add_fwd_ring<TX, S, kEdge, kMode>>(kMaxSmem);
        launch_pdl(add_fwd_ring<TX, S, kEdge, kMode>, p.grid, p.W * p.G, p.smem, st, a, p);
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
