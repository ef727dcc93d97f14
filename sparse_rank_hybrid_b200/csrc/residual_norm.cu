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
// unrounded sum, not of x_out as stored, and the backward recomputes that same sum from x and y (the same
// bytes as reading x_out, and the exact gradient).
//
// Bound by memory: each element is read once and written once (measured DRAM traffic: the algorithm's).  A
// team of threads (the whole block, or a part of a warp for rows of up to 256 channels) owns a row at a time
// and each of its threads the same channels of every row, so the modulation vectors stay in registers for a
// whole modulation row and the sums over tokens are accumulators of the thread.  A worker (team) takes
// consecutive rows; its threads copy the next rows into their own part of a shared-memory ring ahead of the
// arithmetic, so the loads in flight depend neither on registers nor on the barriers of the sums.  The inner
// loop knows nothing of samples and modulation rows: that bookkeeping, a few instructions a row for each of
// six tensors, had cost the backward a fifth (5120 channels: 949 -> 768 us).
//
// B200, back to back, against 6557 GB/s of copy rate: 75,600 x 5120 bf16 forward 0.48-0.52 ms (92-98%),
// backward 0.73-0.79 ms (90-97%); 32,760 x 1536 with an fp32 stream forward 109 us (85%), backward with
// a modulation row per frame and an affine norm 192 us (72%, of which the joining launch takes 10-20).
#include <algorithm>

#include "rows.cuh"

namespace slra {
namespace {

constexpr size_t kRingBytes = 200 * 1024;  // dynamic shared memory of an SM's blocks at most

// Threads of a block at most: the register file holds their coefficients (forward) and also their
// accumulators (backward).  One vector of eight channels a thread as long as the block holds the row (5120
// channels forward: 483 us, with two vectors and half the threads, two blocks an SM, 545), two above.
constexpr int fwd_threads(int V) { return V == 1 ? 1024 : 640; }
constexpr int bwd_threads(int V) { return V == 1 ? 640 : 512; }

// Brings a modulation row towards the SM before the row that needs it.
template <bool SPLIT>
__device__ __forceinline__ void prefetch_mod(const ModTensor& m, int dtype, int b, int f, int column, int gap) {
    if (!m.p) return;
    const int size = dtype == kF32 ? 4 : 2;
    const char* p = static_cast<const char*>(m.p) + (b * m.b + f * m.f + column) * size;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
    if (SPLIT) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + gap * size));
}

// Mean and reciprocal standard deviation from sum(o) and sum(o^2), one barrier for both.  The variance then
// loses a factor 1 + m^2 / var of its digits, so where the mean is more than twice the deviation the caller
// sums the centred row as well (the answer is the same in every thread of the team).
__device__ __forceinline__ bool row_moments(float sum, float squares, float inv, float eps, bool layer, float& m, float& r) {
    m = layer ? sum * inv : 0.f;
    const float var = fmaf(-m, m, squares * inv);
    r = rsqrtf(var + eps);
    return m * m > 4.f * var;
}

// The rows that a team of the grid works on, and where its threads stand in them.
template <bool WIDE>
struct Place {
    int size, t, worker, n, longest, b0, l0;
    __device__ Place(const ResidualNormArgs& a) {
        size = WIDE ? blockDim.x : a.team;
        t = WIDE ? threadIdx.x : threadIdx.x % a.team;
        worker = WIDE ? blockIdx.x : blockIdx.x * (blockDim.x / a.team) + threadIdx.x / a.team;
        const long long r0 = static_cast<long long>(worker) * a.share;
        n = static_cast<int>(min(static_cast<long long>(a.share), max(0ll, a.rows - r0)));
        // teams of one warp take part in each other's shuffles, so they all loop as long as the longest
        longest = WIDE ? n : a.share;
        b0 = static_cast<int>(r0 / a.tokens);
        l0 = static_cast<int>(r0 % a.tokens);
    }
};

// Calls begin(rows), row(valid) for each row, end(rows, done) for every run of a worker's rows within one
// modulation row.  A block-wide team runs through without looking at the row's number; teams that share a
// warp keep in step.
template <bool WIDE, class Begin, class Row, class End>
__device__ __forceinline__ void runs(const Place<WIDE>& at, int per, int first, Begin begin, Row row, End end) {
    if constexpr (WIDE) {
        for (int i = 0; i < at.n;) {
            const int rows = min(per - first, at.n - i);
            begin(rows, i + rows < at.n);
            for (int k = 0; k < rows; ++k) row(true);
            i += rows;
            first = 0;
            end(rows, i);
        }
    } else {
        int rows = 0, left = 0;
        for (int i = 0; i < at.longest; ++i) {
            const bool valid = i < at.n;
            if (valid && left == 0) {
                rows = left = min(per - first, at.n - i);
                first = 0;
                begin(rows, i + rows < at.n);
            }
            row(valid);
            if (valid && --left == 0) end(rows, i + 1);
        }
    }
}

// Y: 0 without y, 1 with it, 2 with its own norm.
template <typename TS, typename TB, int V, int Y, bool WIDE>
__global__ void __launch_bounds__(WIDE ? fwd_threads(V) : 128) residual_norm_fwd_kernel(const __grid_constant__ ResidualNormArgs a) {
    constexpr bool SPLIT = sizeof(TS) == 4;
    constexpr int UX = kUnits<TS>, ONE = UX + (Y ? kUnits<TB> : 0), U = V * ONE;
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float scratch[kTeamScratch];
    const Place<WIDE> at(a);
    Team<WIDE> team(at.size, scratch);
    // first channel, channels between a thread's vectors and between the halves of one
    const int c0 = at.t * (SPLIT ? 4 : 8), step = at.size * (SPLIT ? 4 : 8), gap = SPLIT ? a.channels / 2 : 4;
    const float inv = 1.0f / a.channels;
    const bool layer = a.norm == kNormLayer, scaled = a.rs != 1.f;

    Ring ring(shared_address(shared), a.stages, U);
    bool on[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        on[v] = at.t + v * at.size < a.channels / 8;
        if (!on[v]) ring.clear(v * ONE, ONE);
    }
    RowWalk<const TS> px(a.x, at.b0, at.l0, a.tokens);
    RowWalk<const TB> py(a.y, at.b0, at.l0, a.tokens);
    RowWalk<TS> pxo(a.x_out, at.b0, at.l0, a.tokens);
    RowWalk<TB> ph(a.h, at.b0, at.l0, a.tokens);

    Feed feed(at.n, at.l0, a.tokens);
    auto prefetch = [&]() {
        feed.row([&]() {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!on[v]) continue;
                ring.copy<SPLIT>(v * ONE, px.at(c0 + v * step), gap);
                if (Y) ring.copy<SPLIT>(v * ONE + UX, py.at(c0 + v * step), gap);
            }
        }, [&]() { px.next(), py.next(); }, [&]() { px.wrap(), py.wrap(); });
        ring.filled();
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch();

    Vec cg[V], ca[V], cb[V];  // gate wp, w (1 + scale), b (1 + scale) + shift
#pragma unroll
    for (int v = 0; v < V; ++v) cg[v] = ca[v] = cb[v] = vec_of(0.f);
    int b = at.b0, l = at.l0, f = at.l0 / a.per;

    auto begin = [&](int rows, bool more) {
        const bool last = l + rows == a.tokens;  // the next modulation row is of another sample
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = c0 + v * step;
            if (!on[v]) continue;
            if (Y) {
                const Vec w = load_any<SPLIT>(a.post_weight, c, a.w_dtype, 1.f, gap);
                const Vec g = load_any<SPLIT>(a.gate.p, b * a.gate.b + f * a.gate.f + c, a.mod_dtype, 1.f, gap);
#pragma unroll
                for (int e = 0; e < 4; ++e) cg[v].f[e] = mul2(w.f[e], g.f[e]);
                if (more) prefetch_mod<SPLIT>(a.gate, a.mod_dtype, last ? b + 1 : b, last ? 0 : f + 1, c, gap);
            }
            if (a.norm) {
                const Vec sc = load_any<SPLIT>(a.scale.p, b * a.scale.b + f * a.scale.f + c, a.mod_dtype, 0.f, gap);
                const Vec sh = load_any<SPLIT>(a.shift.p, b * a.shift.b + f * a.shift.f + c, a.mod_dtype, 0.f, gap);
                const Vec w = load_any<SPLIT>(a.weight, c, a.w_dtype, 1.f, gap);
                const Vec bias = load_any<SPLIT>(a.bias, c, a.w_dtype, 0.f, gap);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 up = add2(sc.f[e], both(1.f));
                    ca[v].f[e] = mul2(w.f[e], up);
                    cb[v].f[e] = fma2(bias.f[e], up, sh.f[e]);
                }
                if (more) {
                    prefetch_mod<SPLIT>(a.scale, a.mod_dtype, last ? b + 1 : b, last ? 0 : f + 1, c, gap);
                    prefetch_mod<SPLIT>(a.shift, a.mod_dtype, last ? b + 1 : b, last ? 0 : f + 1, c, gap);
                }
            }
        }
    };
    auto row = [&](bool valid) {
        prefetch();
        ring_wait(a.stages);
        Vec o[V], y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            o[v] = ring.read<TS>(v * ONE);
            if constexpr (Y != 0) y[v] = ring.read<TB>(v * ONE + UX);
        }
        ring.done();
        if constexpr (Y != 0) {
            if constexpr (Y == 2) {
                float2 acc = both(0.f);
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc = fma2(y[v].f[e], y[v].f[e], acc);
                float q[1] = {fold(acc)};
                team.sum(q);
                const float2 ry = both(rsqrtf(q[0] * inv + a.post_eps));
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[v].f[e] = mul2(y[v].f[e], ry);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (scaled) o[v].f[e] = mul2(o[v].f[e], both(a.rs));
                    o[v].f[e] = fma2(cg[v].f[e], y[v].f[e], o[v].f[e]);
                }
                if (valid && on[v]) store_vec<TS, SPLIT>(pxo.at(c0 + v * step), o[v], gap);
            }
            if (valid) pxo.next();
        }
        if (!a.norm) return;
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
            if (valid && on[v]) store_vec<TB, SPLIT>(ph.at(c0 + v * step), o[v], gap);
        }
        if (valid) ph.next();
    };
    auto end = [&](int rows, int) {
        l += rows;
        ++f;
        if (l == a.tokens) {
            l = f = 0;
            ++b;
            pxo.wrap(), ph.wrap();
        }
    };
    runs<WIDE>(at, a.per, l - f * a.per, begin, row, end);
}

template <typename TS, typename TB, int V, int Y, bool WIDE>
__global__ void __launch_bounds__(WIDE ? bwd_threads(V) : 128) residual_norm_bwd_kernel(const __grid_constant__ ResidualNormArgs a) {
    constexpr bool SPLIT = sizeof(TS) == 4;
    constexpr int UX = kUnits<TS>, UB = kUnits<TB>;
    // x, dx_out, dh and y of each vector
    constexpr int DXO = UX, DH = 2 * UX, YU = 2 * UX + UB, ONE = 2 * UX + (Y ? 2 : 1) * UB, U = V * ONE;
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float scratch[kTeamScratch];
    const Place<WIDE> at(a);
    Team<WIDE> team(at.size, scratch);
    const int c0 = at.t * (SPLIT ? 4 : 8), step = at.size * (SPLIT ? 4 : 8), gap = SPLIT ? a.channels / 2 : 4;
    const float inv = 1.0f / a.channels;
    const bool layer = a.norm == kNormLayer, scaled = a.rs != 1.f;
    const bool has_dxo = a.dx_out.p != nullptr, has_dh = a.norm != kNormNone;

    Ring ring(shared_address(shared), a.stages, U);
    bool on[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        on[v] = at.t + v * at.size < a.channels / 8;
        if (!on[v]) ring.clear(v * ONE, ONE);
    }
    RowWalk<const TS> px(a.x, at.b0, at.l0, a.tokens), pdo(a.dx_out, at.b0, at.l0, a.tokens);
    RowWalk<const TB> py(a.y, at.b0, at.l0, a.tokens), pdh(a.dh, at.b0, at.l0, a.tokens);
    RowWalk<TS> pdx(a.dx, at.b0, at.l0, a.tokens);
    RowWalk<TB> pdy(a.dy, at.b0, at.l0, a.tokens);

    Feed feed(at.n, at.l0, a.tokens);
    auto prefetch = [&]() {
        feed.row([&]() {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!on[v]) continue;
                ring.copy<SPLIT>(v * ONE, px.at(c0 + v * step), gap);
                if (has_dxo) ring.copy<SPLIT>(v * ONE + DXO, pdo.at(c0 + v * step), gap);
                if (has_dh) ring.copy<SPLIT>(v * ONE + DH, pdh.at(c0 + v * step), gap);
                if (Y) ring.copy<SPLIT>(v * ONE + YU, py.at(c0 + v * step), gap);
            }
        }, [&]() { px.next(), pdo.next(), pdh.next(), py.next(); }, [&]() { px.wrap(), pdo.wrap(), pdh.wrap(), py.wrap(); });
        ring.filled();
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch();

    Vec cg[V], ca[V];            // gate wp, w (1 + scale)
    Vec p0[V], p1[V], pq[V];     // sums over the rows of a modulation row
#pragma unroll
    for (int v = 0; v < V; ++v) cg[v] = ca[v] = p0[v] = p1[v] = pq[v] = vec_of(0.f);
    // Sums of the weights' gradients over all rows of the worker, added to at the end of each modulation
    // row: this thread's part of shared memory where it has room, else of the worker's slot in wpart.
    // Element e of vector v of sum k is at k wk + v wv + e we (+ wg in the vector's second half).
    float* wslot = a.wpart + static_cast<long long>(at.worker) * 3 * a.channels + c0;
    float* wsum = wslot;
    int wk = a.channels, wv = step, we = 1, wg = gap - 4;
    if (a.wsum_shared) {
        wsum = reinterpret_cast<float*>(shared) + static_cast<size_t>(a.stages) * U * 4 * blockDim.x + threadIdx.x;
        we = blockDim.x, wv = 8 * we, wk = V * wv, wg = 0;
    }
    if (a.wpart)
        for (int v = 0; v < V && on[v]; ++v)
            for (int k = 0; k < 3; ++k)
                for (int e = 0; e < 8; ++e) wsum[k * wk + v * wv + e * we + (e < 4 ? 0 : wg)] = 0.f;
    auto add_weights = [&](int k, int v, int e, float2 d) {  // elements 2e, 2e + 1
        float* w = wsum + k * wk + v * wv + 2 * e * we + (e < 2 ? 0 : wg);
        w[0] += d.x;
        w[we] += d.y;
    };

    int b = at.b0, l = at.l0, f = at.l0 / a.per;
    auto begin = [&](int rows, bool more) {
        const bool last = l + rows == a.tokens;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = c0 + v * step;
            if (!on[v]) continue;
            if (Y) {
                const Vec w = load_any<SPLIT>(a.post_weight, c, a.w_dtype, 1.f, gap);
                const Vec g = load_any<SPLIT>(a.gate.p, b * a.gate.b + f * a.gate.f + c, a.mod_dtype, 1.f, gap);
#pragma unroll
                for (int e = 0; e < 4; ++e) cg[v].f[e] = mul2(w.f[e], g.f[e]);
                if (more) prefetch_mod<SPLIT>(a.gate, a.mod_dtype, last ? b + 1 : b, last ? 0 : f + 1, c, gap);
            }
            const Vec w = load_any<SPLIT>(a.weight, c, a.w_dtype, 1.f, gap);
            const Vec sc = load_any<SPLIT>(a.scale.p, b * a.scale.b + f * a.scale.f + c, a.mod_dtype, 0.f, gap);
#pragma unroll
            for (int e = 0; e < 4; ++e) ca[v].f[e] = fma2(w.f[e], sc.f[e], w.f[e]);
            if (more) prefetch_mod<SPLIT>(a.scale, a.mod_dtype, last ? b + 1 : b, last ? 0 : f + 1, c, gap);
        }
    };
    // Of a row only o stays in registers across a sum; the rest is read again from the ring where it is
    // needed, which costs less than the registers to keep it.
    auto row = [&](bool valid) {
        prefetch();
        ring_wait(a.stages);
        Vec o[V];  // rs x + gate wp yh, then t, the gradient that reaches it
        float2 ry = both(1.f);
        if constexpr (Y == 2) {
            float2 acc = both(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Vec y = ring.read<TB>(v * ONE + YU);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc = fma2(y.f[e], y.f[e], acc);
            }
            float q[1] = {fold(acc)};
            team.sum(q);
            ry = both(rsqrtf(q[0] * inv + a.post_eps));
        }
        float rd = 0.f, mr = 0.f, k1 = 0.f, k0 = 0.f;
        if (has_dh) {
            float2 s1 = both(0.f), s2 = both(0.f), s3 = both(0.f), s4 = both(0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = ring.read<TS>(v * ONE);
                if constexpr (Y != 0) {
                    Vec y = ring.read<TB>(v * ONE + YU);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (Y == 2) y.f[e] = mul2(y.f[e], ry);
                        if (scaled) o[v].f[e] = mul2(o[v].f[e], both(a.rs));
                        o[v].f[e] = fma2(cg[v].f[e], y.f[e], o[v].f[e]);
                    }
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
            float q[4] = {fold(s1), fold(s2), fold(s3), fold(s4)}, m;
            team.sum(q);
            const bool centre = row_moments(q[0], q[1], inv, a.eps, layer, m, rd);
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
                if (centre) rd = rsqrtf(c[0] * inv + a.eps), an = c[1];
            }
            // with n = o rd + mr: rd (a - am - n mean(a n)) = rd a + k1 o + k0
            an *= rd * inv;
            mr = -m * rd;
            k1 = -rd * rd * an;
            k0 = -rd * fmaf(mr, an, am);
        }
        float2 su = both(0.f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Vec d = has_dxo ? ring.read<TS>(v * ONE + DXO) : vec_of(0.f);
            if (has_dh) {
                const Vec dh = ring.read<TB>(v * ONE + DH);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (valid) {
                        p0[v].f[e] = add2(p0[v].f[e], dh.f[e]);
                        p1[v].f[e] = fma2(dh.f[e], fma2(o[v].f[e], both(rd), both(mr)), p1[v].f[e]);
                    }
                    d.f[e] = add2(d.f[e], fma2(o[v].f[e], both(k1), both(k0)));
                    o[v].f[e] = fma2(mul2(dh.f[e], ca[v].f[e]), both(rd), d.f[e]);
                }
            } else {
                o[v] = d;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) d.f[e] = scaled ? mul2(both(a.rs), o[v].f[e]) : o[v].f[e];
            if (valid && on[v]) store_vec<TS, SPLIT>(pdx.at(c0 + v * step), d, gap);
            if constexpr (Y != 0) {
                Vec y = ring.read<TB>(v * ONE + YU);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (Y == 2) y.f[e] = mul2(y.f[e], ry);
                    if (valid) pq[v].f[e] = fma2(o[v].f[e], y.f[e], pq[v].f[e]);
                    o[v].f[e] = mul2(o[v].f[e], cg[v].f[e]);
                    if (Y == 2) su = fma2(o[v].f[e], y.f[e], su);
                }
                if (Y == 1 && valid && on[v]) store_vec<TB, SPLIT>(pdy.at(c0 + v * step), o[v], gap);
            }
        }
        if constexpr (Y == 2) {
            float q[1] = {fold(su)};
            team.sum(q);
            const float2 mu = both(-q[0] * inv * ry.x);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Vec y = ring.read<TB>(v * ONE + YU);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[v].f[e] = mul2(ry, fma2(y.f[e], mu, o[v].f[e]));
                if (valid && on[v]) store_vec<TB, SPLIT>(pdy.at(c0 + v * step), o[v], gap);
            }
        }
        ring.done();
        if (valid) pdx.next(), pdy.next();
    };
    // The end of the modulation row, or of this worker's part of it (`done` of its rows so far): the sums go
    // straight to the gradients where the worker had all its rows, else to the worker's first or last slot.
    auto end = [&](int rows, int done) {
        const bool whole = rows == a.per;
        const long long slot = 2ll * at.worker + (done != rows ? 1 : 0);
        const long long g = (static_cast<long long>(b) * a.groups + f) * a.channels;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = c0 + v * step;
            if (!on[v]) continue;
            if (!whole && a.part) {
                float* part = a.part + slot * 3 * a.channels + c;
                store_vec<float, SPLIT>(part, p0[v], gap);
                store_vec<float, SPLIT>(part + a.channels, p1[v], gap);
                store_vec<float, SPLIT>(part + 2 * a.channels, pq[v], gap);
            }
            if (whole) {
                if (a.dshift) store_vec<float, SPLIT>(a.dshift + g + c, p0[v], gap);
                if (a.dscale) {
                    const Vec w = load_any<SPLIT>(a.weight, c, a.w_dtype, 1.f, gap);
                    const Vec z = load_any<SPLIT>(a.bias, c, a.w_dtype, 0.f, gap);
                    Vec d;
#pragma unroll
                    for (int e = 0; e < 4; ++e) d.f[e] = fma2(w.f[e], p1[v].f[e], mul2(z.f[e], p0[v].f[e]));
                    store_vec<float, SPLIT>(a.dscale + g + c, d, gap);
                }
                if (Y && a.dgate) {
                    Vec d = load_any<SPLIT>(a.post_weight, c, a.w_dtype, 1.f, gap);
#pragma unroll
                    for (int e = 0; e < 4; ++e) d.f[e] = mul2(d.f[e], pq[v].f[e]);
                    store_vec<float, SPLIT>(a.dgate + g + c, d, gap);
                }
            }
            if (a.wpart) {
                const Vec sc = load_any<SPLIT>(a.scale.p, b * a.scale.b + f * a.scale.f + c, a.mod_dtype, 0.f, gap);
                const Vec gt = load_any<SPLIT>(a.gate.p, b * a.gate.b + f * a.gate.f + c, a.mod_dtype, 1.f, gap);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    add_weights(0, v, e, fma2(sc.f[e], p1[v].f[e], p1[v].f[e]));
                    add_weights(1, v, e, fma2(sc.f[e], p0[v].f[e], p0[v].f[e]));
                    if (Y) add_weights(2, v, e, mul2(gt.f[e], pq[v].f[e]));
                }
            }
            p0[v] = p1[v] = pq[v] = vec_of(0.f);
        }
        l += rows;
        ++f;
        if (l == a.tokens) {
            l = f = 0;
            ++b;
            pdx.wrap(), pdy.wrap();
        }
    };
    runs<WIDE>(at, a.per, l - f * a.per, begin, row, end);
    if (a.wpart && a.wsum_shared)
        for (int v = 0; v < V && on[v]; ++v)
            for (int k = 0; k < 3; ++k)
                for (int e = 0; e < 8; ++e)
                    wslot[k * a.channels + v * step + e + (e < 4 ? 0 : gap - 4)] = wsum[k * wk + v * wv + e * we];
}

// The sums over tokens that more than one worker took part in: 32 channels a block, the partial sums
// split over its warps and joined in a fixed order.  Blocks y < jobs join a modulation row's slots (y counts
// modulation rows, or the workers' boundaries where those are fewer), the one after them the weights' sums.
constexpr int kFinalWarps = 16;

__global__ void __launch_bounds__(32 * kFinalWarps) residual_norm_final_kernel(const __grid_constant__ ResidualNormArgs a,
                                                                               int jobs, int by_boundary) {
    __shared__ float red[3][kFinalWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, y = a.wpart ? static_cast<int>(blockIdx.y) - 1 : blockIdx.y;
    const bool in = c < a.channels, weights = y < 0;  // the longest job first
    const int rows = static_cast<int>(a.rows);
    int w0 = 0, w1 = (rows - 1) / a.share, second = -1, g = 0;
    if (!weights) {
        g = y;
        if (by_boundary) {  // the modulation row that worker y + 1's first row continues
            const long long r = (y + 1ll) * a.share;
            g = static_cast<int>(r / a.per);
            if (r >= rows || r == static_cast<long long>(g) * a.per) return;
        }
        const int first = g * a.per;
        w0 = first / a.share;
        w1 = (first + a.per - 1) / a.share;
        if (w0 == w1) return;  // one worker had it all
        // its sums are in the workers' first slots, but in the second one of a worker that came to it from
        // another row
        if (w0 * a.share < first) second = w0;
    }
    float sum[3] = {0.f, 0.f, 0.f};
    if (in) {
        const long long row = 3ll * a.channels;
#pragma unroll 8
        for (int w = w0 + warp; w <= w1; w += kFinalWarps) {
            const float* p = weights ? a.wpart + w * row + c : a.part + (2ll * w + (w == second ? 1 : 0)) * row + c;
#pragma unroll
            for (int k = 0; k < 3; ++k) sum[k] += p[static_cast<long long>(k) * a.channels];
        }
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
        const long long at = static_cast<long long>(g) * a.channels + c;
        if (a.dshift) a.dshift[at] = sum[0];
        if (a.dscale) a.dscale[at] = value(a.weight, 1.f) * sum[1] + value(a.bias, 0.f) * sum[0];
        if (a.dgate) a.dgate[at] = value(a.post_weight, 1.f) * sum[2];
    }
}

// Blocks that an SM holds at once, from the registers the kernels need.
int blocks_per_sm(const RowPlan& p, bool backward) {
    const int threads = backward ? bwd_threads(p.V) : p.V == 1 ? 1024 : 640;  // 96 or 128 registers; 64 or 96
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

template <typename TS, typename TB, int V, int Y, bool WIDE>
cudaError_t launch_dir(ResidualNormArgs a, const RowPlan& p, bool backward, cudaStream_t st) {
    const int units = backward ? 2 * kUnits<TS> + (Y ? 2 : 1) * kUnits<TB> : kUnits<TS> + (Y ? kUnits<TB> : 0);
    const size_t stage = size_t(16) * V * units * p.threads, sums = size_t(3) * V * 32 * p.threads;
    const int per_sm = blocks_per_sm(p, backward);
    const size_t room = kRingBytes / per_sm;
    a.stages = ring_stages(stage, per_sm, room, a.share, 1);
    // the weights' sums take what the ring leaves
    a.wsum_shared = backward && a.wpart && a.stages * stage + sums <= room;
    const size_t smem = a.stages * stage + (a.wsum_shared ? sums : 0);
    return backward ? launch(residual_norm_bwd_kernel<TS, TB, V, Y, WIDE>, a, p, smem, st)
                    : launch(residual_norm_fwd_kernel<TS, TB, V, Y, WIDE>, a, p, smem, st);
}
template <typename TS, typename TB, int V, bool WIDE>
cudaError_t launch_y(const ResidualNormArgs& a, const RowPlan& p, bool backward, cudaStream_t st) {
    return a.y.p == nullptr      ? launch_dir<TS, TB, V, 0, WIDE>(a, p, backward, st)
           : a.post == kNormNone ? launch_dir<TS, TB, V, 1, WIDE>(a, p, backward, st)
                                 : launch_dir<TS, TB, V, 2, WIDE>(a, p, backward, st);
}

template <typename TS, typename TB>
cudaError_t launch_types(const ResidualNormArgs& a, const RowPlan& p, bool backward, cudaStream_t st) {
    return p.team <= 32 ? launch_y<TS, TB, 1, false>(a, p, backward, st)
           : p.V == 1   ? launch_y<TS, TB, 1, true>(a, p, backward, st)
                        : launch_y<TS, TB, 2, true>(a, p, backward, st);
}

}  // namespace

RowPlan residual_norm_plan(long long rows, int channels, bool backward) {
    RowPlan p;
    const int slots = channels / 8;
    row_team(slots, slots > 640 ? 2 : 1, &p);
    row_workers(rows, kSMs * blocks_per_sm(p, backward), &p);
    return p;
}

cudaError_t launch_residual_norm(const ResidualNormArgs& args, bool backward, cudaStream_t st) {
    ResidualNormArgs a = args;
    const RowPlan p = residual_norm_plan(a.rows, a.channels, backward);
    a.team = p.team;
    a.workers = p.workers;
    a.share = p.share;
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
    const bool whole = a.share % a.per == 0 || a.share >= a.rows;  // no modulation row has more than one worker
    const int jobs = a.part && !whole ? static_cast<int>(by_boundary ? p.workers - 1 : mods) : 0;
    const int y = jobs + (a.wpart ? 1 : 0);
    if (y == 0) return cudaSuccess;
    residual_norm_final_kernel<<<dim3((a.channels + 31) / 32, y), 32 * kFinalWarps, 0, st>>>(a, jobs, by_boundary);
    return cudaGetLastError();
}

}  // namespace slra
