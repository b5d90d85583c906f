// addbwd.cuh -- the ring kernel of the residual-stream backwards: dx (with
// the stream's own gradient ds added) and the partial column sums of dw from
// the stream s, or from its 8-bit checkpoint.  addbwd_*.cu instantiate it.
//
// One pass over s (or its codes), dy and ds.  xhat and dn are computed, enter
// the row's sum of dn xhat and the column sums, and after the row reduction
// give dx; they are kept in registers where those suffice and computed a
// second time elsewhere.  A row's rstd and its groups' scales come a row block
// ahead (fed through the ring instead, as two more copies a block, they cost
// 30%).  Measured (bf16, of measured copy bandwidth, graph of passes):
// [16384, 4096] 85 us, 0.93, in every expression (expression 0 with a 16-bit
// weight multiplies packed pairs: 92 us with f32 pairs rounded after); from the
// checkpoint 78 us, 0.89, where unpacking and scaling the codes bounds it; rows
// that start inside a vector 0.55 to 0.8.  Three CTAs an SM at 80 registers,
// reading the row from the ring twice, took 107 us instead of 85.
#pragma once

#include "rowring.cuh"

namespace gbn {
namespace {

template <typename TX, int S, bool kEdge, int kMode>
__global__ void __launch_bounds__(kRow2[S].T, row_minb(kKindB, S))
    add_bwd_ring(const __grid_constant__ BwdArgs a, const __grid_constant__ RowPlan pl)
{
    grid_dependency_sync();
    constexpr int kW = kRow2[S].W, KV = kRow2[S].KV, U = row_U(kKindB, S);
    constexpr int kG = row_G(kKindB, S), kLanes = kW ? kW : 256;
    constexpr int VEC = Vec<TX>::kN, P = VEC / 2, E = (int)sizeof(TX);
    constexpr bool kPacked = kMode == kBwdC || kMode == kBwdInt8, kLean = KV > 2;
    constexpr bool kCast = kMode == kBwdCast, kCast16 = kMode == kBwdCast16;
    constexpr int kType = kMode == kBwdInt8 ? kInt8 : kE4M3;
    // words of a thread's vector of s: activations, or 8-bit codes
    constexpr int NS = kPacked ? VEC / 4 : 4, VS = kPacked ? VEC : 16, ES = kPacked ? 1 : E;
    constexpr int kRed = row_red_floats<kLanes, kG, U, false>();
    extern __shared__ __align__(128) unsigned char dsm[];
    __shared__ float red[kRed];
    int parity = 0;
    const int N = a.N, W = kW ? kW : pl.W, G = kW ? kG : pl.G, R = G * U;
    const int g = threadIdx.x / W, l = threadIdx.x - g * W;
    if constexpr (kW == 0)
        for (int i = threadIdx.x; i < kRed; i += W * G) red[i] = 0.f;
    const int64_t K = row_ring_start(a.in, pl, a.M, dsm);

    int64_t row = (int64_t)blockIdx.x * R + g;  // this thread's first row
    const Cols<VEC, kW, KV, kEdge> cols(l, W, kEdge ? (int)(row * N % VEC) : 0, N);
    f2 wf[KV][P], acc[KV][P];
    load_weights<VEC, kW, KV, kEdge>(wf, cols, a.w, a.wt, a.variant == 2);
    // kCast16 holds the weights as packed pairs: they multiply 16-bit values,
    // and the products are rounded once, as the expression says
    uint32_t wp[KV][P];
    if constexpr (kCast16) {
#pragma unroll
        for (int j = 0; j < KV; ++j)
#pragma unroll
            for (int p = 0; p < P; ++p) wp[j][p] = P16<TX>::from_f2(wf[j][p]);
    }
#pragma unroll
    for (int j = 0; j < KV; ++j)
#pragma unroll
        for (int p = 0; p < P; ++p) acc[j][p] = splat2(0.f);
    int64_t at = row * N - cols.first + l * VEC;
    const int64_t row_step = (int64_t)gridDim.x * R, at_step = row_step * N;
    const uint32_t so0 = pl.off[0] + row_off(a.in[0], kPacked ? 0 : row - g, g) -
                         cols.first * ES + l * VS;
    const uint32_t so1 = pl.off[1] + row_off(a.in[1], row - g, g) - cols.first * E + l * 16;
    const uint32_t so2 = pl.off[2] + row_off(a.in[2], row - g, g) - cols.first * E + l * 16;

    // A row's rstd, and the scale of each vector's group, are loaded one row
    // block ahead of their use.  kEdge: a vector's elements before eb belong to
    // group ga, the others to the next one, whose scale the next lane holds
    // (vectors that span two groups are never a warp's last: groups are aligned
    // runs of lanes, one lane further on; the row's first vector, which starts
    // before it, has ga = -1).
    const bool whole = !kPacked || a.c.shift == 31;
    int ga0 = 0, eb = VEC;
    if (kPacked && !whole) {
        ga0 = cols.col(0) >> a.c.shift;
        if (kEdge) eb = ((ga0 + 1) << a.c.shift) - cols.col(0);
    }
    const int gstep = whole ? 0 : (W * VEC) >> a.c.shift;
    float rs_n[U], sc_n[U][kPacked ? KV : 1];
    auto load_stats = [&](int64_t row0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = row0 + u * G;
            const bool in = r < a.M;
            rs_n[u] = in ? __ldca(a.rstd + r) : 0.f;
            if constexpr (kPacked) {
                const float* const scr = a.c.scale + r * a.c.ng;
#pragma unroll
                for (int j = 0; j < KV; ++j) {
                    const int q = ga0 + j * gstep;
                    sc_n[u][j] = in && q >= 0 && q < a.c.ng ? __ldca(scr + q) : 0.f;
                }
            }
        }
    };
    load_stats(row);

    row_ring(a.in, pl, a.M, dsm, K, [&](int64_t b, const unsigned char* slot, bool alive) {
        const bool last = b == pl.nblocks - 1;
        float rs[U], sc[U][kPacked ? KV : 1], sum[U], none[U];
        bool okr[U];
        // a block of 8-bit rows may start anywhere in a 16-byte unit
        const uint32_t sc0 = kPacked ? ((uint32_t)(b * R) * (uint32_t)N) & 15u : 0u;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            okr[u] = alive && (!last || row + u * G < a.M);
            rs[u] = rs_n[u];
            if constexpr (kPacked) {
#pragma unroll
                for (int j = 0; j < KV; ++j) sc[u][j] = sc_n[u][j] * rs[u];
            }
        }
        auto ld_s = [&](int u, int j, uint32_t (&v)[NS]) {
            const bool ok = okr[u] && cols.ok(j);
            const uint32_t o = so0 + u * G * (uint32_t)a.in[0].row_bytes + j * W * VS;
            if constexpr (kPacked) {
                ld_vec8<VEC>(v, slot, sc0 + o, ok, cols.cut(j), cols.em[j]);
            } else {
                const uint4 q = ld_vec<TX>(slot, o, ok, cols.cut(j), cols.em[j]);
                v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
            }
        };
        auto ld_act = [&](int u, int j, bool present, uint32_t so) {
            const uint32_t o = so + u * G * (uint32_t)a.in[1].row_bytes + j * W * 16;
            return ld_vec<TX>(slot, o, okr[u] && cols.ok(j) && present, cols.cut(j), cols.em[j]);
        };
        uint32_t sp[U][KV][NS];
        uint4 dyp[U][KV], dsp[U][KV];
        if constexpr (!kLean) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < KV; ++j) {
                    ld_s(u, j, sp[u][j]);
                    dyp[u][j] = ld_act(u, j, true, so1);
                    dsp[u][j] = ld_act(u, j, a.in[2].p != nullptr, so2);
                }
        }
        load_stats(row + row_step);
        // xhat, dn and dy of one vector
        auto terms = [&](int u, int j, f2 (&xh)[P], f2 (&dn)[P], f2 (&dv)[P]) {
            if constexpr (kLean) {
                ld_s(u, j, sp[u][j]);
                dyp[u][j] = ld_act(u, j, true, so1);
            }
            if constexpr (kPacked) {
#pragma unroll
                for (int i = 0; i < VEC / 4; ++i)
                    q8_unpack4<kType>(sp[u][j][i], xh[2 * i], xh[2 * i + 1]);
                if constexpr (kEdge) {
                    const float ka = sc[u][j], kb = __shfl_down_sync(0xffffffffu, ka, 1);
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        xh[p] = mul2(xh[p], mk2(2 * p < eb ? ka : kb, 2 * p + 1 < eb ? ka : kb));
                } else {
#pragma unroll
                    for (int p = 0; p < P; ++p) xh[p] = mul2(xh[p], splat2(sc[u][j]));
                }
            } else {
                unpack2<TX>(make_uint4(sp[u][j][0], sp[u][j][1], sp[u][j][2], sp[u][j][3]), xh);
#pragma unroll
                for (int p = 0; p < P; ++p) xh[p] = mul2(xh[p], splat2(rs[u]));
            }
            if constexpr (!kCast16) unpack2<TX>(dyp[u][j], dv);
            if constexpr (kCast16) {
#pragma unroll
                for (int p = 0; p < P; ++p)
                    dn[p] = P16<TX>::to_f2(P16<TX>::mul(word(dyp[u][j], p), wp[j][p]));
                return;
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                dn[p] = mul2(dv[p], wf[j][p]);
                if constexpr (kCast) dn[p] = round2<TX>(dn[p]);
            }
        };
        // xhat and dn are kept over the reduction where they fit the registers
        // (8-bit codes take few), and computed again elsewhere
                constexpr bool kKeep = kPacked && !kEdge && !kLean;
        f2 xk[kKeep ? U : 1][kKeep ? KV : 1][P], dk[kKeep ? U : 1][kKeep ? KV : 1][P];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2 q = splat2(0.f);
#pragma unroll
            for (int j = 0; j < KV; ++j) {
                if (KV > 1 && j >= cols.live) continue;
                f2 (&xh)[P] = xk[kKeep ? u : 0][kKeep ? j : 0];
                f2 (&dn)[P] = dk[kKeep ? u : 0][kKeep ? j : 0];
                f2 dv[P];
                terms(u, j, xh, dn, dv);
#pragma unroll
                for (int p = 0; p < P; ++p) q = fma2(dn[p], xh[p], q);
                // expression 0's term is dy rx(xhat): the exact product, or
                // (kCast16) rounded to x's type
                if constexpr (kCast16) {
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        acc[j][p] = add2(acc[j][p],
                                         P16<TX>::to_f2(P16<TX>::mul(word(dyp[u][j], p),
                                                                     P16<TX>::from_f2(xh[p]))));
                } else if constexpr (kCast) {
#pragma unroll
                    for (int p = 0; p < P; ++p)
                        acc[j][p] = fma2(dv[p], round2<TX>(xh[p]), acc[j][p]);
                } else {
#pragma unroll
                    for (int p = 0; p < P; ++p) acc[j][p] = fma2(dv[p], xh[p], acc[j][p]);
                }
            }
            sum[u] = lo2(q) + hi2(q);
        }
        row_reduce<kLanes, kG, U, false>(sum, none, red, parity, g, l);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const f2 r2 = splat2(rs[u]), nm = splat2(-(sum[u] * a.inv_n));
            TX* const dxr = static_cast<TX*>(a.dx) + at + (int64_t)u * G * N;
#pragma unroll
            for (int j = 0; j < KV; ++j) {
                if (KV > 1 && j >= cols.live) continue;
                f2 (&xh)[P] = xk[kKeep ? u : 0][kKeep ? j : 0];
                f2 (&dn)[P] = dk[kKeep ? u : 0][kKeep ? j : 0];
                f2 dv[P];
                if constexpr (!kKeep) terms(u, j, xh, dn, dv);
                if constexpr (kLean) dsp[u][j] = ld_act(u, j, a.in[2].p != nullptr, so2);
                unpack2<TX>(dsp[u][j], dv);
#pragma unroll
                for (int p = 0; p < P; ++p) dv[p] = fma2(r2, fma2(xh[p], nm, dn[p]), dv[p]);
                st_vec<TX>(dxr + j * W * VEC, pack2<TX>(dv), okr[u] && cols.ok(j), cols.cut(j),
                           cols.em[j]);
            }
        }
        row += row_step;
        at += at_step;
        return kLanes > 32 && !kLean;  // row_reduce's barrier came after the last slot read
    });

    if (a.ws == nullptr) return;  // no weight gradient wanted (uniform)
    // The CTA's column sums, its row groups added in order: each group leaves
    // its vectors in the drained ring, and column c of group q is found
    // `first` of that group's rows further on.
    const int cap = W * KV * VEC;
    float* const out = a.ws + blockIdx.x * (int64_t)N;
    if (G == 1 && !kEdge && (reinterpret_cast<uintptr_t>(out) & 15) == 0) {
#pragma unroll
        for (int j = 0; j < KV; ++j)
            if (cols.ok(j)) {
#pragma unroll
                for (int p = 0; p < P; p += 2)
                    *reinterpret_cast<float4*>(out + cols.col(j) + 2 * p) =
                        make_float4(lo2(acc[j][p]), hi2(acc[j][p]), lo2(acc[j][p + 1]),
                                    hi2(acc[j][p + 1]));
            }
    } else if (G == 1) {
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
                *reinterpret_cast<float2*>(buf + g * cap + cols.vec(j) * VEC + 2 * p) =
                    make_float2(lo2(acc[j][p]), hi2(acc[j][p]));
        __syncthreads();
        for (int c = threadIdx.x; c < N; c += W * G) {
            float t = 0.f;
#pragma unroll 4
            for (int q = 0; q < G; ++q) {
                const int first = kEdge ? (int)(((int64_t)blockIdx.x * R + q) * N % VEC) : 0;
                t += buf[q * cap + c + first];
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
        if constexpr (row_takes(kKindB, S)) {
            ring_attributes<add_bwd_ring<TX, S, kEdge, kMode>>(kMaxSmem);
            launch_pdl(add_bwd_ring<TX, S, kEdge, kMode>, p.grid, p.W * p.G, p.smem, st, a, p);
        }
    };
    auto modes = [&](auto s_, auto edge_) {
        using std::integral_constant;
        if (mode == kBwdC)
            go(s_, edge_, integral_constant<int, kBwdC>{});
        else if (mode == kBwdInt8)
            go(s_, edge_, integral_constant<int, kBwdInt8>{});
        else if (mode == kBwdCast && is16<TX>())
            go(s_, edge_, integral_constant<int, is16<TX>() ? kBwdCast : kBwdS>{});
        else if (mode == kBwdCast16 && is16<TX>())
            go(s_, edge_, integral_constant<int, is16<TX>() ? kBwdCast16 : kBwdS>{});
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
