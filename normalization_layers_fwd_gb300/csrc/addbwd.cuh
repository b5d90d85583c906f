// addbwd.cuh -- the ring kernel of the residual-stream backwards: dx (with
// the stream's own gradient ds added) and the partial column sums of dw from
// the stream s, or from its 8-bit checkpoint.  addbwd_*.cu instantiate it.
#pragma once

#include "rowring.cuh"

namespace gbn {
namespace {

// VEC 8-bit codes as floats.
template <int VEC>
__device__ __forceinline__ void unpack_vec8(const uint32_t (&v)[VEC / 4], f2 (&o)[VEC / 2], int type)
{
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        o[2 * i] = q8_unpack2(v[i] & 0xffffu, type);
        o[2 * i + 1] = q8_unpack2(v[i] >> 16, type);
    }
}

template <typename TX, int S, bool kEdge, int kMode>
__global__ void __launch_bounds__(kRow[S].T, bwd_minb(S))
    add_bwd_ring(const __grid_constant__ BwdArgs a, const __grid_constant__ RowPlan pl)
{
    grid_dependency_sync();
    constexpr int W = kRow[S].W, T = kRow[S].T, KV = kRow[S].KV, U = row_U(S), G = T / W;
    constexpr int VEC = Vec<TX>::kN, P = VEC / 2, E = (int)sizeof(TX);
    constexpr bool kPacked = kMode == kBwdC, kCast = kMode == kBwdCast;
    // words of a thread's vector of s: activations, or 8-bit codes
    constexpr int NS = kPacked ? VEC / 4 : 4, ES = kPacked ? 1 : E;
    extern __shared__ __align__(128) unsigned char dsm[];
    __shared__ float red[row_red_floats<W, T, U, false>()];
    int parity = 0;
    const int N = a.N, g = threadIdx.x / W, l = threadIdx.x % W;
    const int64_t K = row_ring_start(a.in, pl, a.M, dsm);
    const int64_t first_row = (int64_t)blockIdx.x * pl.R + g;
    const Cols<VEC, W, KV, kEdge> cols(l, kEdge ? (int)(first_row * N % VEC) : 0, N);
    f2 wf[KV][P], acc[KV][P];
    load_weights<VEC, W, KV, kEdge>(wf, cols, a.w, a.wt, a.variant == 2);
#pragma unroll
    for (int j = 0; j < KV; ++j)
#pragma unroll
        for (int p = 0; p < P; ++p) acc[j][p] = splat2(0.f);
    // expression 0 with a weight of x's type rounds each term of dw
    const bool round_terms = kCast && a.wt == dtype_code<TX>();

    // A row's rstd, and the scales of its vectors' groups, are loaded one row
    // block ahead of their use.  kEdge: elements from eb on take the second.
    int ga[KV], eb[KV];
    if constexpr (kPacked)
#pragma unroll
        for (int j = 0; j < KV; ++j) {
            const int c = cols.col(j) < 0 ? 0 : cols.col(j);
            const bool whole = a.c.shift == 31;
            ga[j] = whole ? 0 : c >> a.c.shift;
            eb[j] = kEdge && !whole ? ((ga[j] + 1) << a.c.shift) - cols.col(j) : VEC;
        }
    constexpr int kSc = kPacked ? (kEdge ? 2 : 1) : 0;
    float rs_n[U], sc_n[U][KV][kSc ? kSc : 1];
    auto load_stats = [&](int64_t row0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = row0 + u * G;
            const bool ok = r < a.M;
            rs_n[u] = ok ? __ldca(a.rstd + r) : 0.f;
            if constexpr (kPacked) {
#pragma unroll
                for (int j = 0; j < KV; ++j) {
                    const float* sc = a.c.scale + r * a.c.ng + ga[j];
                    const bool in = ok && cols.ok(j);
                    sc_n[u][j][0] = in ? __ldca(sc) : 0.f;
                    if constexpr (kEdge)
                        sc_n[u][j][1] =
                            in && eb[j] < VEC && ga[j] + 1 < a.c.ng ? __ldca(sc + 1) : 0.f;
                }
            }
        }
    };
    load_stats(first_row);

    row_ring(a.in, pl, a.M, dsm, K, [&](int64_t b, const unsigned char* slot, bool alive) {
        const int64_t r0 = b * pl.R;
        const bool last = b == pl.nblocks - 1;
        uint32_t sp[U][KV][NS];
        uint4 dyp[U][KV], dsp[U][KV];
        float rs[U], sc[U][KV][kSc ? kSc : 1], sum[U], none[U];
        bool okr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = g + u * G;
            const int64_t r = r0 + i;
            okr[u] = alive && r < a.M;
            rs[u] = rs_n[u];
            const uint32_t o0 = row_off(a.in[0], r0, i) - cols.first * ES;
            const uint32_t o1 = row_off(a.in[1], r0, i) - cols.first * E;
            const uint32_t o2 = row_off(a.in[2], r0, i) - cols.first * E;
#pragma unroll
            for (int j = 0; j < KV; ++j) {
                const bool ok = okr[u] && cols.ok(j);
                const int v = l + j * W;
                const int64_t at = r * N - cols.first + (int64_t)v * VEC;
                if constexpr (kPacked) {
                    ld_vec8<VEC, kEdge>(sp[u][j], slot + pl.off[0], o0 + v * VEC, ok, a.in[0],
                                        last, at, cols.em[j]);
#pragma unroll
                    for (int q = 0; q < kSc; ++q) sc[u][j][q] = sc_n[u][j][q];
                } else {
                    const uint4 q = ld_vec<TX, kEdge>(slot + pl.off[0], o0 + v * 16, ok, a.in[0],
                                                      last, at * E, cols.em[j]);
                    sp[u][j][0] = q.x, sp[u][j][1] = q.y, sp[u][j][2] = q.z, sp[u][j][3] = q.w;
                }
                dyp[u][j] = ld_vec<TX, kEdge>(slot + pl.off[1], o1 + v * 16, ok, a.in[1], last,
                                              at * E, cols.em[j]);
                dsp[u][j] = ld_vec<TX, kEdge>(slot + pl.off[2], o2 + v * 16, ok && a.in[2].p,
                                              a.in[2], last, at * E, cols.em[j]);
            }
        }
        load_stats(r0 + (int64_t)gridDim.x * pl.R + g);
        // xhat and dn of one vector
        auto terms = [&](int u, int j, f2 (&xh)[P], f2 (&dn)[P], f2 (&dv)[P]) {
            if constexpr (kPacked) {
                unpack_vec8<VEC>(sp[u][j], xh, a.c.type);
                const float ka = sc[u][j][0] * rs[u];
                if constexpr (kEdge) {
                    const float kb = sc[u][j][kSc - 1] * rs[u];
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        xh[p] = mul2(xh[p], mk2(2 * p < eb[j] ? ka : kb,
                                                2 * p + 1 < eb[j] ? ka : kb));
                } else {
#pragma unroll
                    for (int p = 0; p < P; ++p) xh[p] = mul2(xh[p], splat2(ka));
                }
            } else {
                unpack2<TX>(make_uint4(sp[u][j][0], sp[u][j][1], sp[u][j][2], sp[u][j][3]), xh);
#pragma unroll
                for (int p = 0; p < P; ++p) xh[p] = mul2(xh[p], splat2(rs[u]));
            }
            unpack2<TX>(dyp[u][j], dv);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                dn[p] = mul2(dv[p], wf[j][p]);
                if constexpr (kCast) dn[p] = round2<TX>(dn[p]);
            }
        };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2 q = splat2(0.f);
#pragma unroll
            for (int j = 0; j < KV; ++j) {
                f2 xh[P], dn[P], dv[P];
                terms(u, j, xh, dn, dv);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    q = fma2(dn[p], xh[p], q);
                    if constexpr (kCast) {
                        // the term dy rx(xhat): its product is exact in float32, rounded to
                        // x's type when the weight has that type
                        f2 t = mul2(dv[p], round2<TX>(xh[p]));
                        if (round_terms) t = round2<TX>(t);
                        acc[j][p] = add2(acc[j][p], t);
                    } else {
                        acc[j][p] = fma2(dv[p], xh[p], acc[j][p]);
                    }
                }
            }
            sum[u] = lo2(q) + hi2(q);
        }
        row_reduce<W, T, U, false>(sum, none, red, parity);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + g + u * G;
            const f2 r2 = splat2(rs[u]), nm = splat2(-(sum[u] * a.inv_n));
            TX* const dxr = static_cast<TX*>(a.dx) + (r * N - cols.first);
#pragma unroll
            for (int j = 0; j < KV; ++j) {
                f2 xh[P], dn[P], dv[P];
                terms(u, j, xh, dn, dv);
                unpack2<TX>(dsp[u][j], dv);
#pragma unroll
                for (int p = 0; p < P; ++p) dv[p] = fma2(r2, fma2(xh[p], nm, dn[p]), dv[p]);
                st_vec<TX, kEdge>(dxr + (l + j * W) * VEC, pack2<TX>(dv), okr[u] && cols.ok(j),
                                  cols.em[j]);
            }
        }
        return W > 32;  // row_reduce's barrier came after the last slot read
    });

    if (a.ws == nullptr) return;  // no weight gradient wanted (uniform)
    // The CTA's column sums, its row groups added in order: each group leaves
    // its vectors in the drained ring, and column c of group q is found
    // `first` of that group's rows further on.
    constexpr int kCap = W * KV * VEC;
    float* const out = a.ws + blockIdx.x * (int64_t)N;
    if constexpr (G == 1) {
#pragma unroll
        for (int j = 0; j < KV; ++j)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int c = cols.col(j) + 2 * p;
                if ((cols.em[j] >> (2 * p)) & 1u) out[c] = lo2(acc[j][p]);
                if ((cols.em[j] >> (2 * p + 1)) & 1u) out[c + 1] = hi2(acc[j][p]);
            }
    } else {
        float* const buf = reinterpret_cast<float*>(dsm + 128);
#pragma unroll
        for (int j = 0; j < KV; ++j)
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<float2*>(buf + g * kCap + (l + j * W) * VEC + 2 * p) =
                    make_float2(lo2(acc[j][p]), hi2(acc[j][p]));
        __syncthreads();
        for (int c = threadIdx.x; c < N; c += T) {
            float t = 0.f;
#pragma unroll 4
            for (int q = 0; q < G; ++q) {
                const int first =
                    kEdge ? (int)(((int64_t)blockIdx.x * pl.R + q) * N % VEC) : 0;
                t += buf[q * kCap + c + first];
            }
            out[c] = t;
        }
    }
}

template <typename TX>
cudaError_t bwd_launch(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p)
{
    auto go = [&](auto s_, auto edge_, auto mode_) {
        constexpr int S = decltype(s_)::value, kMode = decltype(mode_)::value;
        constexpr bool kEdge = decltype(edge_)::value;
        ring_attributes<add_bwd_ring<TX, S, kEdge, kMode>>(kMaxSmem);
        launch_pdl(add_bwd_ring<TX, S, kEdge, kMode>, p.grid, kRow[S].T, p.smem, st, a, p);
    };
    auto modes = [&](auto s_, auto edge_) {
        using std::integral_constant;
        if (mode == kBwdC)
            go(s_, edge_, integral_constant<int, kBwdC>{});
        else if (mode == kBwdCast && is16<TX>())
            go(s_, edge_, integral_constant<int, is16<TX>() ? kBwdCast : kBwdS>{});
        else
            go(s_, edge_, integral_constant<int, kBwdS>{});
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
