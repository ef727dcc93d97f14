// Gated residual and modulated norm in one pass over the rows (tokens), and its gradient.
//
//   forward   yh = y, or y rsqrt(mean(y^2) + e') with the norm behind the block
//             o  = rs x + gate wp yh
//             h  = (o - m) r w (1 + scale) + b (1 + scale) + shift,  r = rsqrt(mean((o - m)^2) + e),
//             m = mean(o) (LAYER) or 0 (RMS)
//   backward  a = dh w (1 + scale), n = (o - m) r
//             t = dx_out + r (a - mean(a) [LAYER] - n mean(a n)),  dx = rs t
//             u = t gate wp,  dy = u, or ry (u - yh mean(u yh)) with the norm behind the block
//             per modulation row (sample, frame or token): P0 = sum dh, P1 = sum dh n, Q = sum t yh,
//             from which dshift = P0, dscale = w P1 + b P0, dgate = wp Q, and over all modulation rows
//             dw = sum (1 + scale) P1, db = sum (1 + scale) P0, dwp = sum gate Q.
//
// Everything is computed in fp32 from the inputs and rounded once on the way out: h is the norm of the
// unrounded sum, not of x_out as stored, and the backward recomputes that same sum from x and y.  The
// variance is a second sum over the centred row, which stays in registers, so a mean far from zero costs
// no digits.
//
// Bound by memory: each element is read once and written once.  A team of threads (the whole block, or a
// part of a warp for narrow rows) owns a row at a time and each of its threads the same columns of every
// row, so the modulation vectors stay in registers for a whole modulation row and the sums over tokens
// are per-thread accumulators.  A worker (team) takes consecutive rows; its threads copy the next rows
// into their own part of a shared-memory ring ahead of the arithmetic, so the loads in flight do not
// depend on registers or on the barriers of the sums.
#include <algorithm>

#include "rows.cuh"

namespace slra {
namespace {

constexpr size_t kRingBytes = 200 * 1024;  // dynamic shared memory of an SM's blocks at most

// Threads of a block at most: the register file holds their coefficients (forward) and also their
// accumulators (backward).
constexpr int fwd_threads(int V) { return V == 1 ? 1024 : 640; }
constexpr int bwd_threads(int V) { return V == 1 ? 640 : 512; }

// A pointer that walks a worker's rows through a [B][L][C] tensor with free batch and token strides.
template <typename T>
struct RowWalk {
    T* p;
    __device__ RowWalk(const RowTensor& t, int b, int l, int column)
        : p(static_cast<T*>(t.p) + b * t.b + l * t.l + column) {}
    __device__ __forceinline__ void next(const RowTensor& t) { p += t.l; }
    __device__ __forceinline__ void wrap(const RowTensor& t, int tokens) { p += t.b - tokens * t.l; }
};

// Brings a modulation row towards the SM before the row that needs it.
__device__ __forceinline__ void prefetch_mod(const ModTensor& m, int dtype, int b, int f, int column) {
    if (m.p)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(m.p) +
                                                      (b * m.b + f * m.f + column) * (dtype == kF32 ? 4 : 2)));
}

// Mean and reciprocal standard deviation from sum(o) and sum(o^2).  One pass over the row loses a factor
// 1 + m^2 / var of the digits, so where the mean is more than twice the deviation the caller sums the
// centred row instead (the same answer in every thread of the team).
__device__ __forceinline__ bool row_moments(float sum, float squares, float inv, float eps, bool layer, float& m, float& r) {
    m = layer ? sum * inv : 0.f;
    const float var = fmaf(-m, m, squares * inv);
    r = rsqrtf(var + eps);
    return m * m > 4.f * var;
}

template <typename TS, typename TB, int V, bool HASY, bool WIDE>
__global__ void __launch_bounds__(WIDE ? fwd_threads(V) : 128) residual_norm_fwd_kernel(const __grid_constant__ ResidualNormArgs a) {
    constexpr int UX = kUnits<TS>, UY = HASY ? kUnits<TB> : 0, U = V * (UX + UY);
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float scratch[kTeamScratch];
    const int team_size = WIDE ? blockDim.x : a.team;
    Team<WIDE> team(team_size, scratch);
    const int t = WIDE ? threadIdx.x : threadIdx.x % a.team;
    const int worker = WIDE ? blockIdx.x : blockIdx.x * (blockDim.x / a.team) + threadIdx.x / a.team;
    const long long r0 = worker_lo(a.rows, a.workers, worker), r1 = worker_lo(a.rows, a.workers, worker + 1);
    const int n = static_cast<int>(r1 - r0);
    // teams of one warp take part in each other's shuffles, so they all loop as long as the longest
    const int iters = WIDE ? n : static_cast<int>((a.rows + a.workers - 1) / a.workers);
    const int b0 = static_cast<int>(r0 / a.tokens), l0 = static_cast<int>(r0 % a.tokens), c0 = t * 8;
    const int step = team_size * 8;  // channels between a thread's vectors
    const float inv = 1.0f / a.channels;
    const bool layer = a.norm == kNormLayer;

    Ring ring(shared_address(shared), a.stages, U);
    bool on[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        on[v] = c0 + v * step < a.channels;
        if (!on[v]) ring.clear(v * (UX + UY), UX + UY);
    }
    RowWalk<const TS> px(a.x, b0, l0, c0);
    RowWalk<const TB> py(HASY ? a.y : a.h, b0, l0, c0);
    RowWalk<TS> pxo(HASY ? a.x_out : a.x, b0, l0, c0);
    RowWalk<TB> ph(a.norm ? a.h : a.y, b0, l0, c0);

    int lp = l0, left = n;  // token of the next row to copy, rows still to copy
    auto prefetch = [&]() {
        if (left > 0) {
            --left;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!on[v]) continue;
                ring.copy(v * (UX + UY), px.p + v * step);
                if (HASY) ring.copy(v * (UX + UY) + UX, py.p + v * step);
            }
            px.next(a.x);
            if (HASY) py.next(a.y);
            if (++lp == a.tokens) {
                lp = 0;
                px.wrap(a.x, a.tokens);
                if (HASY) py.wrap(a.y, a.tokens);
            }
            ring.filled();
        }
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch();

    Vec cg[V], ca[V], cb[V];  // gate wp, w (1 + scale), b (1 + scale) + shift
#pragma unroll
    for (int v = 0; v < V; ++v) cg[v] = ca[v] = cb[v] = vec_of(0.f);
    int b = b0, l = l0, f = l0 / a.per, group_left = 0;
    for (int i = 0; i < iters; ++i) {
        prefetch();
        const bool row = WIDE || i < n;
        if (row && group_left == 0) {  // another modulation row
            group_left = a.per - (l - f * a.per);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = c0 + v * step;
                if (!on[v]) continue;
                if (HASY) {
                    const Vec w = load_any(a.post_weight, c, a.w_dtype, 1.f);
                    const Vec g = load_any(a.gate.p, b * a.gate.b + f * a.gate.f + c, a.mod_dtype, 1.f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) cg[v].f[e] = mul2(w.f[e], g.f[e]);
                }
                if (a.norm) {
                    const Vec sc = load_any(a.scale.p, b * a.scale.b + f * a.scale.f + c, a.mod_dtype, 0.f);
                    const Vec sh = load_any(a.shift.p, b * a.shift.b + f * a.shift.f + c, a.mod_dtype, 0.f);
                    const Vec w = load_any(a.weight, c, a.w_dtype, 1.f), bias = load_any(a.bias, c, a.w_dtype, 0.f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 up = add2(sc.f[e], both(1.f));
                        ca[v].f[e] = mul2(w.f[e], up);
                        cb[v].f[e] = fma2(bias.f[e], up, sh.f[e]);
                    }
                }
            }
        }
        if (row && group_left == 1 && i + 1 < n) {  // the next row's modulation
            const bool wrap = l + 1 == a.tokens;
            const int nb = wrap ? b + 1 : b, nf = wrap ? 0 : f + 1;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = c0 + v * step;
                if (!on[v]) continue;
                if (HASY) prefetch_mod(a.gate, a.mod_dtype, nb, nf, c);
                prefetch_mod(a.scale, a.mod_dtype, nb, nf, c);
                prefetch_mod(a.shift, a.mod_dtype, nb, nf, c);
            }
        }
        ring_wait(a.stages);
        Vec o[V], y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            o[v] = ring.read<TS>(v * (UX + UY));
            if (HASY) y[v] = ring.read<TB>(v * (UX + UY) + UX);
        }
        ring.done();

        if (HASY) {
            if (a.post) {
                float q[1] = {0.f};
                float2 acc = both(0.f);
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc = fma2(y[v].f[e], y[v].f[e], acc);
                q[0] = fold(acc);
                team.sum(q);
                const float2 ry = both(rsqrtf(q[0] * inv + a.post_eps));
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[v].f[e] = mul2(y[v].f[e], ry);
            }
            const float2 rs = both(a.rs);
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[v].f[e] = fma2(cg[v].f[e], y[v].f[e], mul2(rs, o[v].f[e]));
                if (row && on[v]) store_vec(pxo.p + v * step, o[v]);
            }
        }
        if (a.norm) {
            float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s1 = add2(s1, o[v].f[e]);
                    s2 = fma2(o[v].f[e], o[v].f[e], s2);
                }
            float q[2] = {fold(s1), fold(s2)}, m, r;
            team.sum(q);
            const bool centre = row_moments(q[0], q[1], inv, a.eps, layer, m, r);
            if (WIDE ? centre : __any_sync(0xffffffffu, centre)) {  // every team of a warp takes part in the sum
                float c[1] = {0.f};
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 d = add2(o[v].f[e], both(-m));
                        if (on[v]) c[0] += fold(mul2(d, d));
                    }
                team.sum(c);
                if (centre) r = rsqrtf(c[0] * inv + a.eps);
            }
            const float2 rr = both(r), mr = both(-m * r);
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[v].f[e] = fma2(fma2(o[v].f[e], rr, mr), ca[v].f[e], cb[v].f[e]);
                if (row && on[v]) store_vec(ph.p + v * step, o[v]);
            }
        }
        if (row) {
            --group_left;
            ++l;
            if (HASY) pxo.next(a.x_out);
            if (a.norm) ph.next(a.h);
            if (group_left == 0) ++f;
            if (l == a.tokens) {
                l = f = 0;
                ++b;
                if (HASY) pxo.wrap(a.x_out, a.tokens);
                if (a.norm) ph.wrap(a.h, a.tokens);
            }
        }
    }
}

template <typename TS, typename TB, int V, bool HASY, bool WIDE>
__global__ void __launch_bounds__(WIDE ? bwd_threads(V) : 128) residual_norm_bwd_kernel(const __grid_constant__ ResidualNormArgs a) {
    constexpr int UX = kUnits<TS>, UB = kUnits<TB>;
    constexpr int ONE = 2 * UX + (HASY ? 2 : 1) * UB, U = V * ONE;  // x, dx_out, dh and y of each vector
    constexpr int DXO = UX, DH = 2 * UX, Y = 2 * UX + UB;
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float scratch[kTeamScratch];
    const int team_size = WIDE ? blockDim.x : a.team;
    Team<WIDE> team(team_size, scratch);
    const int t = WIDE ? threadIdx.x : threadIdx.x % a.team;
    const int worker = WIDE ? blockIdx.x : blockIdx.x * (blockDim.x / a.team) + threadIdx.x / a.team;
    const long long r0 = worker_lo(a.rows, a.workers, worker), r1 = worker_lo(a.rows, a.workers, worker + 1);
    const int n = static_cast<int>(r1 - r0);
    const int iters = WIDE ? n : static_cast<int>((a.rows + a.workers - 1) / a.workers);
    const int b0 = static_cast<int>(r0 / a.tokens), l0 = static_cast<int>(r0 % a.tokens), c0 = t * 8;
    const int step = team_size * 8;
    const float inv = 1.0f / a.channels;
    const bool layer = a.norm == kNormLayer, has_dxo = a.dx_out.p != nullptr, has_dh = a.norm != kNormNone;

    Ring ring(shared_address(shared), a.stages, U);
    bool on[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        on[v] = c0 + v * step < a.channels;
        if (!on[v]) ring.clear(v * ONE, ONE);
    }
    RowWalk<const TS> px(a.x, b0, l0, c0), pdo(a.dx_out, b0, l0, c0);
    RowWalk<const TB> py(a.y, b0, l0, c0), pdh(a.dh, b0, l0, c0);
    RowWalk<TS> pdx(a.dx, b0, l0, c0);
    RowWalk<TB> pdy(a.dy, b0, l0, c0);

    int lp = l0, left = n;
    auto prefetch = [&]() {
        if (left > 0) {
            --left;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!on[v]) continue;
                ring.copy(v * ONE, px.p + v * step);
                if (has_dxo) ring.copy(v * ONE + DXO, pdo.p + v * step);
                if (has_dh) ring.copy(v * ONE + DH, pdh.p + v * step);
                if (HASY) ring.copy(v * ONE + Y, py.p + v * step);
            }
            px.next(a.x);
            pdo.next(a.dx_out);
            pdh.next(a.dh);
            if (HASY) py.next(a.y);
            if (++lp == a.tokens) {
                lp = 0;
                px.wrap(a.x, a.tokens);
                pdo.wrap(a.dx_out, a.tokens);
                pdh.wrap(a.dh, a.tokens);
                if (HASY) py.wrap(a.y, a.tokens);
            }
            ring.filled();
        }
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch();

    Vec cg[V], ca[V];            // gate wp, w (1 + scale)
    Vec p0[V], p1[V], pq[V];     // sums over the rows of a modulation row
#pragma unroll
    for (int v = 0; v < V; ++v) cg[v] = ca[v] = p0[v] = p1[v] = pq[v] = vec_of(0.f);
    // Sums of the weights' gradients over all rows of the worker, added to at the end of each modulation
    // row: this thread's part of shared memory where it has room, else of the worker's slot in wpart.
    float* wslot = a.wpart + static_cast<long long>(worker) * 3 * a.channels + c0;
    float* wsum = wslot;
    int wk = a.channels, wv = step, we = 1;  // strides of the sum, the vector and the element
    if (a.wsum_shared) {
        wsum = reinterpret_cast<float*>(shared) + static_cast<size_t>(a.stages) * U * 4 * blockDim.x + threadIdx.x;
        we = blockDim.x, wv = 8 * we, wk = V * wv;
    }
    if (a.wpart)
        for (int v = 0; v < V && c0 + v * step < a.channels; ++v)
            for (int k = 0; k < 3; ++k)
                for (int e = 0; e < 8; ++e) wsum[k * wk + v * wv + e * we] = 0.f;

    int b = b0, l = l0, f = l0 / a.per, group_left = 0, seg_rows = 0;
    for (int i = 0; i < iters; ++i) {
        prefetch();
        const bool row = WIDE || i < n;
        if (row && group_left == 0) {
            group_left = a.per - (l - f * a.per);
            seg_rows = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = c0 + v * step;
                if (!on[v]) continue;
                if (HASY) {
                    const Vec w = load_any(a.post_weight, c, a.w_dtype, 1.f);
                    const Vec g = load_any(a.gate.p, b * a.gate.b + f * a.gate.f + c, a.mod_dtype, 1.f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) cg[v].f[e] = mul2(w.f[e], g.f[e]);
                }
                const Vec w = load_any(a.weight, c, a.w_dtype, 1.f);
                const Vec sc = load_any(a.scale.p, b * a.scale.b + f * a.scale.f + c, a.mod_dtype, 0.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) ca[v].f[e] = fma2(w.f[e], sc.f[e], w.f[e]);
            }
        }
        if (row && group_left == 1 && i + 1 < n) {
            const bool wrap = l + 1 == a.tokens;
            const int nb = wrap ? b + 1 : b, nf = wrap ? 0 : f + 1;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = c0 + v * step;
                if (!on[v]) continue;
                if (HASY) prefetch_mod(a.gate, a.mod_dtype, nb, nf, c);
                prefetch_mod(a.scale, a.mod_dtype, nb, nf, c);
            }
        }
        ring_wait(a.stages);
        Vec o[V];
        float2 ry = both(1.f);
        if (HASY && a.post) {
            float2 acc = both(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Vec y = ring.read<TB>(v * ONE + Y);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc = fma2(y.f[e], y.f[e], acc);
            }
            float q[1] = {fold(acc)};
            team.sum(q);
            ry = both(rsqrtf(q[0] * inv + a.post_eps));
        }
        // o: the sum rs x + gate wp yh, then t, the gradient that reaches it; the other rows are read again
        // from the ring where they are needed, which costs less than the registers to keep them
        float2 rr = both(0.f), mr = both(0.f), c0r = both(0.f), c1r = both(0.f);
        if (has_dh) {
            const float2 rs = both(a.rs);
            float2 s1 = both(0.f), s2 = both(0.f), s3 = both(0.f), s4 = both(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = ring.read<TS>(v * ONE);
                if (HASY) {
                    const Vec y = ring.read<TB>(v * ONE + Y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[v].f[e] = fma2(cg[v].f[e], mul2(y.f[e], ry), mul2(rs, o[v].f[e]));
                }
                const Vec dh = ring.read<TB>(v * ONE + DH);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 d = mul2(dh.f[e], ca[v].f[e]);
                    s1 = add2(s1, o[v].f[e]);
                    s2 = fma2(o[v].f[e], o[v].f[e], s2);
                    s3 = add2(s3, d);
                    s4 = fma2(o[v].f[e], d, s4);
                }
            }
            float q[4] = {fold(s1), fold(s2), fold(s3), fold(s4)}, m, r;
            team.sum(q);
            const bool centre = row_moments(q[0], q[1], inv, a.eps, layer, m, r);
            const float am = layer ? q[2] * inv : 0.f;
            float an = fmaf(-m, q[2], q[3]);  // sum of a (o - m)
            if (WIDE ? centre : __any_sync(0xffffffffu, centre)) {
                float c[2] = {0.f, 0.f};
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (!on[v]) continue;
                    const Vec dh = ring.read<TB>(v * ONE + DH);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 d = add2(o[v].f[e], both(-m));
                        c[0] += fold(mul2(d, d));
                        c[1] += fold(mul2(d, mul2(dh.f[e], ca[v].f[e])));
                    }
                }
                team.sum(c);
                if (centre) r = rsqrtf(c[0] * inv + a.eps), an = c[1];
            }
            an *= r * inv;  // mean(a n)
            // r (a - am - n an) = r a + c1 o + c0 with n = o r - m r
            rr = both(r), mr = both(-m * r);
            c1r = both(-r * r * an), c0r = both(r * (m * r * an - am));
        }
        float2 su = both(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Vec d = has_dxo ? ring.read<TS>(v * ONE + DXO) : vec_of(0.f);
            if (has_dh) {
                const Vec dh = ring.read<TB>(v * ONE + DH);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (row) {
                        const float2 nrm = fma2(o[v].f[e], rr, mr);
                        p0[v].f[e] = add2(p0[v].f[e], dh.f[e]);
                        p1[v].f[e] = fma2(dh.f[e], nrm, p1[v].f[e]);
                    }
                    const float2 step_o = fma2(o[v].f[e], c1r, c0r);
                    o[v].f[e] = add2(d.f[e], fma2(mul2(dh.f[e], ca[v].f[e]), rr, step_o));
                }
            } else {
                o[v] = d;
            }
            const float2 rs = both(a.rs);
#pragma unroll
            for (int e = 0; e < 4; ++e) d.f[e] = mul2(rs, o[v].f[e]);
            if (row && on[v]) store_vec(pdx.p + v * step, d);
            if (HASY) {
                const Vec y = ring.read<TB>(v * ONE + Y);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 yh = mul2(y.f[e], ry);
                    if (row) pq[v].f[e] = fma2(o[v].f[e], yh, pq[v].f[e]);
                    o[v].f[e] = mul2(o[v].f[e], cg[v].f[e]);
                    if (a.post) su = fma2(o[v].f[e], yh, su);
                }
                if (!a.post && row && on[v]) store_vec(pdy.p + v * step, o[v]);
            }
        }
        if (HASY && a.post) {
            float q[1] = {fold(su)};
            team.sum(q);
            const float2 mu = both(-q[0] * inv * ry.x);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Vec y = ring.read<TB>(v * ONE + Y);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[v].f[e] = mul2(ry, fma2(y.f[e], mu, o[v].f[e]));
                if (row && on[v]) store_vec(pdy.p + v * step, o[v]);
            }
        }
        ring.done();
        if (row) {
            ++seg_rows;
            if (group_left == 1 || i + 1 == n) {
                // end of the modulation row, or of this worker's part of it: the sums go straight to the
                // gradients where the worker had all its rows, else to the worker's first or last slot
                const bool whole = seg_rows == a.per;
                const long long slot = 2ll * worker + (i + 1 != seg_rows ? 1 : 0);
                const long long g = (static_cast<long long>(b) * a.groups + f) * a.channels;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = c0 + v * step;
                    if (!on[v]) continue;
                    if (!whole && a.part) {
                        float* part = a.part + slot * 3 * a.channels + c;
                        store_vec(part, p0[v]);
                        store_vec(part + a.channels, p1[v]);
                        store_vec(part + 2 * a.channels, pq[v]);
                    }
                    if (whole) {
                        if (a.dshift) store_vec(a.dshift + g + c, p0[v]);
                        if (a.dscale) {
                            const Vec w = load_any(a.weight, c, a.w_dtype, 1.f), z = load_any(a.bias, c, a.w_dtype, 0.f);
                            Vec d;
#pragma unroll
                            for (int e = 0; e < 4; ++e) d.f[e] = fma2(w.f[e], p1[v].f[e], mul2(z.f[e], p0[v].f[e]));
                            store_vec(a.dscale + g + c, d);
                        }
                        if (HASY && a.dgate) {
                            Vec d = load_any(a.post_weight, c, a.w_dtype, 1.f);
#pragma unroll
                            for (int e = 0; e < 4; ++e) d.f[e] = mul2(d.f[e], pq[v].f[e]);
                            store_vec(a.dgate + g + c, d);
                        }
                    }
                    if (a.wpart) {
                        float* ws = wsum + v * wv;
                        const Vec sc = load_any(a.scale.p, b * a.scale.b + f * a.scale.f + c, a.mod_dtype, 0.f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 d1 = fma2(sc.f[e], p1[v].f[e], p1[v].f[e]), d0 = fma2(sc.f[e], p0[v].f[e], p0[v].f[e]);
                            ws[2 * e * we] += d1.x, ws[(2 * e + 1) * we] += d1.y;
                            ws[wk + 2 * e * we] += d0.x, ws[wk + (2 * e + 1) * we] += d0.y;
                        }
                        if (HASY) {
                            const Vec gt = load_any(a.gate.p, b * a.gate.b + f * a.gate.f + c, a.mod_dtype, 1.f);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 d = mul2(gt.f[e], pq[v].f[e]);
                                ws[2 * wk + 2 * e * we] += d.x, ws[2 * wk + (2 * e + 1) * we] += d.y;
                            }
                        }
                    }
                    p0[v] = p1[v] = pq[v] = vec_of(0.f);
                }
            }
            --group_left;
            ++l;
            pdx.next(a.dx);
            if (HASY) pdy.next(a.dy);
            if (group_left == 0) ++f;
            if (l == a.tokens) {
                l = f = 0;
                ++b;
                pdx.wrap(a.dx, a.tokens);
                if (HASY) pdy.wrap(a.dy, a.tokens);
            }
        }
    }
    if (a.wpart && a.wsum_shared)
        for (int v = 0; v < V && c0 + v * step < a.channels; ++v)
            for (int k = 0; k < 3; ++k)
                for (int e = 0; e < 8; ++e) wslot[k * a.channels + v * step + e] = wsum[k * wk + v * wv + e * we];
}

// The sums over tokens that more than one worker took part in: 32 channels a block, the partial sums
// split over its 16 warps and joined in a fixed order.  Blocks y < groups join a modulation row's slots
// (y counts modulation rows, or the workers' boundaries where those are fewer), the last one the
// weights' sums.
constexpr int kFinalWarps = 16;

__global__ void __launch_bounds__(32 * kFinalWarps) residual_norm_final_kernel(const __grid_constant__ ResidualNormArgs a,
                                                                               int jobs, int by_boundary) {
    __shared__ float red[3][kFinalWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const bool in = c < a.channels;
    const bool weights = static_cast<int>(blockIdx.y) == jobs;
    int w0 = 0, w1 = a.workers - 1;
    long long g = 0;
    if (!weights) {
        g = blockIdx.y;
        if (by_boundary) {  // the modulation row that worker y + 1's first row continues
            const long long r = worker_lo(a.rows, a.workers, static_cast<int>(blockIdx.y) + 1);
            g = r / a.per;
            if (g * a.per == r || r == a.rows) return;
        }
        w0 = worker_of(a.rows, a.workers, g * a.per);
        w1 = worker_of(a.rows, a.workers, (g + 1) * a.per - 1);
        if (w0 == w1) return;
    }
    float sum[3] = {0.f, 0.f, 0.f};
    if (in)
        for (int w = w0 + warp; w <= w1; w += kFinalWarps) {
            const float* p;
            if (weights) {
                p = a.wpart + static_cast<long long>(w) * 3 * a.channels + c;
            } else {
                if (worker_lo(a.rows, a.workers, w) == worker_lo(a.rows, a.workers, w + 1)) continue;
                const int last = worker_lo(a.rows, a.workers, w) < g * a.per ? 1 : 0;
                p = a.part + (2ll * w + last) * 3 * a.channels + c;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) sum[k] += p[static_cast<long long>(k) * a.channels];
        }
#pragma unroll
    for (int k = 0; k < 3; ++k) red[k][warp][lane] = sum[k];
    __syncthreads();
    if (warp != 0 || !in) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        sum[k] = 0.f;
        for (int w = 0; w < kFinalWarps; ++w) sum[k] += red[k][w][lane];
    }
    auto value = [&](const void* p, float fill) {
        if (!p) return fill;
        if (a.w_dtype == kF32) return static_cast<const float*>(p)[c];
        if (a.w_dtype == kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]);
        return __half2float(static_cast<const __half*>(p)[c]);
    };
    if (weights) {
        if (a.dweight) a.dweight[c] = sum[0];
        if (a.dbias) a.dbias[c] = sum[1];
        if (a.dpost) a.dpost[c] = sum[2];
    } else {
        const long long at = g * a.channels + c;
        if (a.dshift) a.dshift[at] = sum[0];
        if (a.dscale) a.dscale[at] = value(a.weight, 1.f) * sum[1] + value(a.bias, 0.f) * sum[0];
        if (a.dgate) a.dgate[at] = value(a.post_weight, 1.f) * sum[2];
    }
}

// Blocks that a processor holds at once, from the registers the kernels need.
int blocks_per_sm(const RowPlan& p, bool backward) {
    const int threads = backward ? bwd_threads(p.V) : p.V == 1 ? 1024 : 640;
    return std::max(1, threads / p.threads);
}

template <typename K>
cudaError_t launch(K kernel, const ResidualNormArgs& a, const RowPlan& p, size_t smem, cudaStream_t st) {
    if (smem > 40 * 1024) {  // 48 KB without opting in, less the static part
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    kernel<<<p.blocks, p.threads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename TS, typename TB, int V, bool WIDE>
cudaError_t launch_dir(ResidualNormArgs a, const RowPlan& p, bool backward, cudaStream_t st) {
    const bool y = a.y.p != nullptr;
    const int units = backward ? 2 * kUnits<TS> + (y ? 2 : 1) * kUnits<TB> : kUnits<TS> + (y ? kUnits<TB> : 0);
    const size_t stage = size_t(16) * V * units * p.threads, sums = size_t(3) * V * 32 * p.threads;
    const int per_sm = blocks_per_sm(p, backward);
    const size_t room = kRingBytes / per_sm;
    a.stages = ring_stages(stage, per_sm, room);
    // the weights' sums take what the ring leaves
    a.wsum_shared = backward && a.wpart && a.stages * stage + sums <= room;
    const size_t smem = a.stages * stage + (a.wsum_shared ? sums : 0);
    if (!backward)
        return y ? launch(residual_norm_fwd_kernel<TS, TB, V, true, WIDE>, a, p, smem, st)
                 : launch(residual_norm_fwd_kernel<TS, TB, V, false, WIDE>, a, p, smem, st);
    return y ? launch(residual_norm_bwd_kernel<TS, TB, V, true, WIDE>, a, p, smem, st)
             : launch(residual_norm_bwd_kernel<TS, TB, V, false, WIDE>, a, p, smem, st);
}

template <typename TS, typename TB>
cudaError_t launch_types(const ResidualNormArgs& a, const RowPlan& p, bool backward, cudaStream_t st) {
    return p.team <= 32 ? launch_dir<TS, TB, 1, false>(a, p, backward, st)
           : p.V == 1   ? launch_dir<TS, TB, 1, true>(a, p, backward, st)
                        : launch_dir<TS, TB, 2, true>(a, p, backward, st);
}

}  // namespace

// One vector of eight channels a thread, or two: see blocks_per_sm.
RowPlan residual_norm_plan(long long rows, int channels, bool backward) {
    RowPlan p;
    const int slots = channels / 8;
    row_team(slots, slots > (backward ? bwd_threads(1) : 384) ? 2 : 1, &p);
    row_workers(rows, kSMs * blocks_per_sm(p, backward), &p);
    return p;
}

cudaError_t launch_residual_norm(const ResidualNormArgs& args, bool backward, cudaStream_t st) {
    ResidualNormArgs a = args;
    const RowPlan p = residual_norm_plan(a.rows, a.channels, backward);
    a.team = p.team;
    a.workers = p.workers;
    cudaError_t e;
    if (a.stream_dtype == kF32)
        e = a.block_dtype == kF32    ? launch_types<float, float>(a, p, backward, st)
            : a.block_dtype == kBf16 ? launch_types<float, __nv_bfloat16>(a, p, backward, st)
                                     : launch_types<float, __half>(a, p, backward, st);
    else if (a.stream_dtype == kBf16)
        e = launch_types<__nv_bfloat16, __nv_bfloat16>(a, p, backward, st);
    else
        e = launch_types<__half, __half>(a, p, backward, st);
    if (e != cudaSuccess || !backward) return e;
    const long long mods = a.rows / a.per;
    const int by_boundary = mods > p.workers ? 1 : 0;
    const int jobs = a.part ? static_cast<int>(by_boundary ? p.workers - 1 : mods) : 0;
    const int y = jobs + (a.wpart ? 1 : 0);
    if (y == 0) return cudaSuccess;
    residual_norm_final_kernel<<<dim3((a.channels + 31) / 32, y), 32 * kFinalWarps, 0, st>>>(a, jobs, by_boundary);
    return cudaGetLastError();
}

}  // namespace slra
