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
// Where every row has its own modulation vectors (TOKEN: per-token modulation, single tokens) those would be
// loaded and waited for in each row: they travel through the ring with it instead, their gradients are written
// as the row is, and the accumulators hold the weights' sums (60,983 x 392 with an fp32 stream, backward with an
// affine norm: 676 -> 200 us), even where the ring then has one stage only.  One stage of the widest rows, all in fp32, always fits (192 KB).
//
// B200, back to back, against 6557 GB/s of copy rate, over cards and places of the buffers: 75,600 x 5120 bf16
// forward 0.48-0.52 ms (91-99%), backward 0.73-0.85 ms (83-97%); 32,760 x 1536 with an fp32 stream forward
// 108-110 us (84-85%), backward with a modulation row per frame and an affine norm 184-189 us (73-75%), with the
// norm behind the block 165 us (84%), with vectors for each token 343 us (94%).
#pragma once

#include <algorithm>

#include "rows.cuh"

namespace slra {
namespace {

constexpr size_t kRingBytes = 200 * 1024;  // dynamic shared memory of an SM's blocks at most

// Threads of a block at most: the register file holds their coefficients (forward) and also their
// accumulators (backward).  One vector of eight channels a thread as long as the block holds the row (5120
// channels forward: 483 us, with two vectors and half the threads, two blocks an SM, 545), two above.
constexpr int fwd_threads(int V) { return V == 1 ? 1024 : 640; }
// Backward, with the norm behind the block (`sums`: three dependent sums a row) more warps on fewer registers hide
// more than those cost (47,250 x 2048 affine: 298 us with 640 threads, 271 with 768; 30,990 x 2 x 2696 fp32 stream
// 714 and 587), without it they hide less (47,250 x 2048: 204 and 222), nor with vectors for each row (683 and 873).
constexpr int bwd_threads(int V, bool sums) { return V > 1 ? 512 : sums ? 768 : 640; }
// Blocks an SM for rows that share a block of 128 threads.
constexpr int kFwdNarrow = 5, kBwdNarrow = 4;

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

// Rows with a modulation row each: there is nothing to begin or end.
template <bool WIDE, class Row>
__device__ __forceinline__ void each_row(const Place<WIDE>& at, Row row) {
    for (int i = 0; i < at.longest; ++i) row(WIDE || i < at.n);
}

// The sum over a block's teams (each `size` lanes of its four warps) of a thread's four values, in a fixed
// order, in the threads of the first team.
constexpr int kJoinScratch = 4 * 128;  // floats of shared memory
__device__ __forceinline__ float4 join_teams(float4 u, int size, float* scratch) {
    for (int o = size; o < 32; o *= 2) {
        u.x += __shfl_xor_sync(0xffffffffu, u.x, o), u.y += __shfl_xor_sync(0xffffffffu, u.y, o);
        u.z += __shfl_xor_sync(0xffffffffu, u.z, o), u.w += __shfl_xor_sync(0xffffffffu, u.w, o);
    }
    float4* s = reinterpret_cast<float4*>(scratch);
    s[threadIdx.x] = u;
    __syncthreads();
    const int t = threadIdx.x & 31;
    float4 sum = s[t];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
        const float4 p = s[w * 32 + t];
        sum.x += p.x, sum.y += p.y, sum.z += p.z, sum.w += p.w;
    }
    __syncthreads();
    return sum;
}

// The modulation vectors of rows that have one each (TOKEN), and the weights: copies of each thread's channels
// in its part of shared memory, the former in the ring behind the row's own units, the latter behind the ring.
// Vector v of tensor k is at unit (k V + v) u; u units of 16 bytes hold eight elements.
struct ModWalk {
    const char* p;         // moves on where there is no such tensor too: ask the tensor
    long long step, back;  // as RowWalk's
    __device__ ModWalk(const ModTensor& m, int size, int b, int l, int tokens)
        : p(static_cast<const char*>(m.p) + (b * m.b + l * m.f) * size),
          step(m.f * size), back((m.b - tokens * m.f) * size) {}
    __device__ __forceinline__ void next() { p += step; }
    __device__ __forceinline__ void wrap() { p += back; }
};
template <bool SPLIT>
__device__ __forceinline__ void copy_any(uint32_t smem, uint32_t unit, const char* p, int dtype, int column, int gap) {
    if (dtype == kF32) {
        async_copy16(smem, p + column * 4);
        async_copy16(smem + unit, p + (column + (SPLIT ? gap : 4)) * 4);
    } else if (SPLIT) {
        async_copy8(smem, p + column * 2);
        async_copy8(smem + 8, p + (column + gap) * 2);
    } else {
        async_copy16(smem, p + column * 2);
    }
}
__device__ __forceinline__ Vec read_any(uint32_t smem, uint32_t unit, int dtype) {
    if (dtype == kF32) {
        const uint4 u[2] = {shared16(smem), shared16(smem + unit)};
        return unpack<float>(u);
    }
    const uint4 u[1] = {shared16(smem)};
    return dtype == kBf16 ? unpack<__nv_bfloat16>(u) : unpack<__half>(u);
}

// Y: 0 without y, 1 with it, 2 with its own norm.  TOKEN: every row has its own modulation vectors.
template <typename TS, typename TB, int V, int Y, bool WIDE, bool TOKEN>
__global__ void __launch_bounds__(WIDE ? fwd_threads(V) : 128, WIDE ? 1 : kFwdNarrow) residual_norm_fwd_kernel(const __grid_constant__ ResidualNormArgs a) {
    constexpr bool SPLIT = sizeof(TS) == 4;
    constexpr int UX = kUnits<TS>, ONE = UX + (Y ? kUnits<TB> : 0), U = V * ONE;  // units of a row: x and y of each vector
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float scratch[kTeamScratch];
    const Place<WIDE> at(a);
    Team<WIDE> team(at.size, scratch);
    // first channel, channels between a thread's vectors and between the halves of one
    const int c0 = at.t * (SPLIT ? 4 : 8), step = at.size * (SPLIT ? 4 : 8), gap = SPLIT ? a.channels / 2 : 4;
    const float inv = 1.0f / a.channels;
    const bool layer = a.norm == kNormLayer, scaled = a.rs != 1.f;

    const int MU = TOKEN ? a.mod_units : 0, WU = TOKEN ? a.weight_units : 0;
    Ring ring(shared_address(shared), a.stages, U + (Y ? 3 : 2) * V * MU);
    bool on[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        on[v] = at.t + v * at.size < a.channels / 8;
        if (!on[v]) ring.clear(v * ONE, ONE);
    }
    const int mod_size = a.mod_dtype == kF32 ? 4 : 2;
    ModWalk psc(a.scale, mod_size, at.b0, at.l0, a.tokens), psh(a.shift, mod_size, at.b0, at.l0, a.tokens);
    ModWalk pg(a.gate, mod_size, at.b0, at.l0, a.tokens);
    const uint32_t wbase = ring.last + ring.stage;
    if (TOKEN && WU) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!on[v]) continue;
            const void* const w[3] = {a.weight, a.bias, a.post_weight};
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (w[k])
                    copy_any<SPLIT>(wbase + (k * V + v) * WU * ring.unit, ring.unit, static_cast<const char*>(w[k]),
                                    a.w_dtype, c0 + v * step, gap);
        }
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
                if (TOKEN) {
                    const uint32_t m = ring.in + (U + v * MU) * ring.unit, next = V * MU * ring.unit;
                    if (a.scale.p) copy_any<SPLIT>(m, ring.unit, psc.p, a.mod_dtype, c0 + v * step, gap);
                    if (a.shift.p) copy_any<SPLIT>(m + next, ring.unit, psh.p, a.mod_dtype, c0 + v * step, gap);
                    if (Y && a.gate.p) copy_any<SPLIT>(m + 2 * next, ring.unit, pg.p, a.mod_dtype, c0 + v * step, gap);
                }
            }
        }, [&]() {
            px.next(), py.next();
            if (TOKEN) psc.next(), psh.next(), pg.next();
        }, [&]() {
            px.wrap(), py.wrap();
            if (TOKEN) psc.wrap(), psh.wrap(), pg.wrap();
        });
        ring.filled();
        async_commit();
    };
    // A stage of rows with vectors of their own is large: filled again as soon as it is read, one more row is in
    // flight.  41,854 x 4624 fp16 with fp32 vectors, affine: without y 825 -> 583 us, with y and its norm 1219 ->
    // 968, not affine 836 and 838; up to 6% slower at 1536 channels and below.  Other rows: 720p 515 -> 555.
    for (int s = 0; s < a.stages - (TOKEN ? 0 : 1); ++s) prefetch();

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
        if (!TOKEN) prefetch();
        ring_wait(a.stages);
        Vec o[V], y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            o[v] = ring.read<TS>(v * ONE);
            if constexpr (Y != 0) y[v] = ring.read<TB>(v * ONE + UX);
            if (TOKEN && on[v]) {
                const uint32_t m = ring.out + (U + v * MU) * ring.unit, next = V * MU * ring.unit;
                const uint32_t w = wbase + v * WU * ring.unit, wnext = V * WU * ring.unit;
                if (Y) {
                    cg[v] = a.gate.p ? read_any(m + 2 * next, ring.unit, a.mod_dtype) : vec_of(1.f);
                    if (a.post_weight) {
                        const Vec u = WU ? read_any(w + 2 * wnext, ring.unit, a.w_dtype) : load_any<SPLIT>(a.post_weight, c0 + v * step, a.w_dtype, 1.f, gap);
#pragma unroll
                        for (int e = 0; e < 4; ++e) cg[v].f[e] = mul2(u.f[e], cg[v].f[e]);
                    }
                }
                ca[v] = vec_of(1.f);
                if (a.scale.p) {
                    const Vec u = read_any(m, ring.unit, a.mod_dtype);
#pragma unroll
                    for (int e = 0; e < 4; ++e) ca[v].f[e] = add2(u.f[e], both(1.f));
                }
                cb[v] = a.shift.p ? read_any(m + next, ring.unit, a.mod_dtype) : vec_of(0.f);
                if (a.bias) {
                    const Vec u = WU ? read_any(w + wnext, ring.unit, a.w_dtype) : load_any<SPLIT>(a.bias, c0 + v * step, a.w_dtype, 0.f, gap);
#pragma unroll
                    for (int e = 0; e < 4; ++e) cb[v].f[e] = fma2(u.f[e], ca[v].f[e], cb[v].f[e]);
                }
                if (a.weight) {
                    const Vec u = WU ? read_any(w, ring.unit, a.w_dtype) : load_any<SPLIT>(a.weight, c0 + v * step, a.w_dtype, 1.f, gap);
#pragma unroll
                    for (int e = 0; e < 4; ++e) ca[v].f[e] = mul2(u.f[e], ca[v].f[e]);
                }
            }
        }
        ring.done();
        if (TOKEN) prefetch();
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
    if constexpr (TOKEN)
        each_row(at, [&](bool valid) {
            row(valid);
            if (valid && ++l == a.tokens) l = 0, pxo.wrap(), ph.wrap();
        });
    else
        runs<WIDE>(at, a.per, l - f * a.per, begin, row, end);
}

template <typename TS, typename TB, int V, int Y, bool WIDE, bool TOKEN>
__global__ void __launch_bounds__(WIDE ? bwd_threads(V, Y == 2 && !TOKEN) : 128, WIDE ? 1 : kBwdNarrow) residual_norm_bwd_kernel(const __grid_constant__ ResidualNormArgs a) {
    constexpr bool SPLIT = sizeof(TS) == 4;
    constexpr int UX = kUnits<TS>, UB = kUnits<TB>;
    // x, dx_out, dh and y of each vector
    constexpr int DXO = UX, DH = 2 * UX, YU = 2 * UX + UB, ONE = 2 * UX + (Y ? 2 : 1) * UB, U = V * ONE;
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float scratch[WIDE ? kTeamScratch : kJoinScratch];
    const Place<WIDE> at(a);
    Team<WIDE> team(at.size, scratch);
    const int c0 = at.t * (SPLIT ? 4 : 8), step = at.size * (SPLIT ? 4 : 8), gap = SPLIT ? a.channels / 2 : 4;
    const float inv = 1.0f / a.channels;
    const bool layer = a.norm == kNormLayer, scaled = a.rs != 1.f;
    const bool has_dxo = a.dx_out.p != nullptr, has_dh = a.norm != kNormNone;

    const int MU = TOKEN ? a.mod_units : 0, WU = TOKEN ? a.weight_units : 0;
    Ring ring(shared_address(shared), a.stages, U + (Y ? 2 : 1) * V * MU);
    bool on[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        on[v] = at.t + v * at.size < a.channels / 8;
        if (!on[v]) ring.clear(v * ONE, ONE);
    }
    const int mod_size = a.mod_dtype == kF32 ? 4 : 2;
    ModWalk psc(a.scale, mod_size, at.b0, at.l0, a.tokens), pg(a.gate, mod_size, at.b0, at.l0, a.tokens);
    const uint32_t wbase = ring.last + ring.stage;
    if (TOKEN && WU) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!on[v]) continue;
            const void* const w[3] = {a.weight, a.bias, a.post_weight};
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (w[k])
                    copy_any<SPLIT>(wbase + (k * V + v) * WU * ring.unit, ring.unit, static_cast<const char*>(w[k]),
                                    a.w_dtype, c0 + v * step, gap);
        }
    }
    long long grad_at = (static_cast<long long>(at.b0) * a.tokens + at.l0) * a.channels;  // TOKEN: of the row's gradients
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
                if (TOKEN) {
                    const uint32_t m = ring.in + (U + v * MU) * ring.unit;
                    if (a.scale.p) copy_any<SPLIT>(m, ring.unit, psc.p, a.mod_dtype, c0 + v * step, gap);
                    if (Y && a.gate.p) copy_any<SPLIT>(m + V * MU * ring.unit, ring.unit, pg.p, a.mod_dtype, c0 + v * step, gap);
                }
            }
        }, [&]() {
            px.next(), pdo.next(), pdh.next(), py.next();
            if (TOKEN) psc.next(), pg.next();
        }, [&]() {
            px.wrap(), pdo.wrap(), pdh.wrap(), py.wrap();
            if (TOKEN) psc.wrap(), pg.wrap();
        });
        ring.filled();
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch();

    Vec cg[V], ca[V];            // gate wp, w (1 + scale)
    Vec p0[V], p1[V], pq[V];     // sums over the rows of a modulation row
#pragma unroll
    for (int v = 0; v < V; ++v) cg[v] = ca[v] = p0[v] = p1[v] = pq[v] = vec_of(0.f);
    // Sums of the weights' gradients over all rows of the worker.  TOKEN: p0, p1, pq themselves.  Else added to
    // at the end of each modulation row: this thread's part of shared memory where it has room, else of the
    // worker's slot in wpart.  Half i of vector v of sum k is at k wk + v wv + i wi.
    float* const wslot = a.wpart + static_cast<long long>(at.worker) * 3 * a.channels + c0;
    float* wsum = wslot;
    int wk = a.channels, wv = step, wi = gap;
    if (!TOKEN && a.wsum_shared) {
        wsum = reinterpret_cast<float*>(shared) + (static_cast<size_t>(a.stages) * U * blockDim.x + threadIdx.x) * 4;
        wi = 4 * blockDim.x, wv = 2 * wi, wk = V * wv;
    }
    if (!TOKEN && a.wpart)
        for (int v = 0; v < V && on[v]; ++v)
            for (int k = 0; k < 3; ++k)
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<float4*>(wsum + k * wk + v * wv + i * wi) = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add_weights = [&](int k, int v, const Vec& d) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float4* w = reinterpret_cast<float4*>(wsum + k * wk + v * wv + i * wi);
            float4 u = *w;
            u.x += d.f[2 * i].x, u.y += d.f[2 * i].y, u.z += d.f[2 * i + 1].x, u.w += d.f[2 * i + 1].y;
            *w = u;
        }
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
        const auto mod = [&](int k, int v) {  // TOKEN: this row's scale, gate
            const uint32_t m = ring.out + (U + (k * V + v) * MU) * ring.unit;
            return (k ? a.gate.p : a.scale.p) ? read_any(m, ring.unit, a.mod_dtype) : vec_of(k ? 1.f : 0.f);
        };
        const auto weight = [&](int k, int v) {  // weight, bias, post_weight
            const void* w = k == 0 ? a.weight : k == 1 ? a.bias : a.post_weight;
            if (!WU || !w) return load_any<SPLIT>(w, c0 + v * step, a.w_dtype, k == 1 ? 0.f : 1.f, gap);
            return read_any(wbase + (k * V + v) * WU * ring.unit, ring.unit, a.w_dtype);
        };
        if (TOKEN) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!on[v]) continue;
                if (Y) {
                    const Vec g = mod(1, v), w = weight(2, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) cg[v].f[e] = mul2(w.f[e], g.f[e]);
                }
                const Vec sc = mod(0, v), w = weight(0, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) ca[v].f[e] = fma2(w.f[e], sc.f[e], w.f[e]);
            }
        }
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
                if (TOKEN && valid && on[v]) {
                    Vec dn;  // the row's own gradients, and with 1 + scale its part of the weights'
#pragma unroll
                    for (int e = 0; e < 4; ++e) dn.f[e] = mul2(dh.f[e], fma2(o[v].f[e], both(rd), both(mr)));
                    if (a.dshift) store_vec<float, SPLIT>(a.dshift + grad_at + c0 + v * step, dh, gap);
                    if (a.dscale) {
                        const Vec w = weight(0, v), z = weight(1, v);
                        Vec ds;
#pragma unroll
                        for (int e = 0; e < 4; ++e) ds.f[e] = fma2(w.f[e], dn.f[e], mul2(z.f[e], dh.f[e]));
                        store_vec<float, SPLIT>(a.dscale + grad_at + c0 + v * step, ds, gap);
                    }
                    if (a.wpart) {
                        const Vec sc = mod(0, v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 up = add2(sc.f[e], both(1.f));
                            p0[v].f[e] = fma2(up, dh.f[e], p0[v].f[e]);
                            p1[v].f[e] = fma2(up, dn.f[e], p1[v].f[e]);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!TOKEN && valid) {
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
                if (TOKEN && valid && on[v] && (a.dgate || a.wpart)) {
                    Vec dg;
#pragma unroll
                    for (int e = 0; e < 4; ++e) dg.f[e] = mul2(o[v].f[e], Y == 2 ? mul2(y.f[e], ry) : y.f[e]);
                    if (a.wpart) {
                        const Vec g = mod(1, v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) pq[v].f[e] = fma2(g.f[e], dg.f[e], pq[v].f[e]);
                    }
                    if (a.dgate) {
                        const Vec w = weight(2, v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) dg.f[e] = mul2(w.f[e], dg.f[e]);
                        store_vec<float, SPLIT>(a.dgate + grad_at + c0 + v * step, dg, gap);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (Y == 2) y.f[e] = mul2(y.f[e], ry);
                    if (!TOKEN && valid) pq[v].f[e] = fma2(o[v].f[e], y.f[e], pq[v].f[e]);
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
        if (valid) pdx.next(), pdy.next(), grad_at += a.channels;
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
                    p1[v].f[e] = fma2(sc.f[e], p1[v].f[e], p1[v].f[e]);
                    p0[v].f[e] = fma2(sc.f[e], p0[v].f[e], p0[v].f[e]);
                    pq[v].f[e] = mul2(gt.f[e], pq[v].f[e]);
                }
                add_weights(0, v, p1[v]);
                add_weights(1, v, p0[v]);
                if (Y) add_weights(2, v, pq[v]);
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
    if constexpr (TOKEN)
        each_row(at, [&](bool valid) {
            row(valid);
            if (valid && ++l == a.tokens) l = 0, pdx.wrap(), pdy.wrap();
        });
    else
        runs<WIDE>(at, a.per, l - f * a.per, begin, row, end);
    launch_dependents();
    if (!a.wpart || (WIDE && wsum == wslot && !TOKEN)) return;
    // A block's slot: its first worker's.
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
                if (on[v]) {
                    if constexpr (TOKEN) {
                        const Vec& d = k == 0 ? p1[v] : k == 1 ? p0[v] : pq[v];
                        u = make_float4(d.f[2 * i].x, d.f[2 * i].y, d.f[2 * i + 1].x, d.f[2 * i + 1].y);
                    } else {
                        u = *reinterpret_cast<const float4*>(wsum + k * wk + v * wv + i * wi);
                    }
                }
                if (!WIDE) u = join_teams(u, at.size, scratch);
                if (on[v] && (WIDE || threadIdx.x < at.size))
                    *reinterpret_cast<float4*>(wslot + k * a.channels + v * step + i * gap) = u;
            }
}

// Blocks that an SM holds at once, from the registers the kernels need.
inline int blocks_per_sm(const RowPlan& p, bool backward) {
    if (p.team <= 32) return backward ? kBwdNarrow : kFwdNarrow;
    return std::max(1, (backward ? bwd_threads(p.V, p.sums) : fwd_threads(p.V)) / p.threads);
}

template <typename K>
cudaError_t launch(K kernel, const ResidualNormArgs& a, const RowPlan& p, size_t smem, cudaStream_t st) {
    const cudaError_t e = allow_shared(kernel, smem, kRingBytes);
    if (e != cudaSuccess) return e;
    kernel<<<p.blocks, p.threads, smem, st>>>(a);
    return cudaGetLastError();
}

// Dynamic shared memory of a block: the ring, then the weights (TOKEN) or their gradients' sums.
struct RowShared {
    int stages, mod_units, weight_units, wsum;
    size_t bytes;
};
inline RowShared row_shared(const ResidualNormArgs& a, const RowPlan& p, bool backward, bool token) {
    const int ts = a.stream_dtype == kF32 ? 2 : 1, tb = a.block_dtype == kF32 ? 2 : 1, y = a.y.p ? 1 : 0;
    const size_t unit = size_t(16) * p.V * p.threads;
    size_t units = backward ? 2 * ts + (1 + y) * tb : ts + y * tb;
    RowShared s{};
    const int per_sm = blocks_per_sm(p, backward);
    size_t room = kRingBytes / per_sm, weights = 0;
    if (token) {
        s.mod_units = !a.gate.p && !a.scale.p && !a.shift.p ? 0 : a.mod_dtype == kF32 ? 2 : 1;
        s.weight_units = !a.weight && !a.bias && !a.post_weight ? 0 : a.w_dtype == kF32 ? 2 : 1;
        units += ((backward ? 1 : 2) + y) * s.mod_units;
    }
    s.stages = ring_stages(units * unit, per_sm, room, a.share, 1, token && !backward);
    if (token) {  // the weights too, if the ring keeps its stages
        weights = 3 * s.weight_units * unit;
        if (s.stages * units * unit + weights > room) s.weight_units = 0, weights = 0;
    }
    // the sums take what the ring leaves
    if (backward && !token && a.wpart && (s.stages * units + 6) * unit <= room) s.wsum = 1, weights = 6 * unit;
    s.bytes = s.stages * units * unit + weights;
    return s;
}

template <typename TS, typename TB, int V, int Y, bool WIDE, bool BACKWARD, bool TOKEN>
cudaError_t launch_dir(ResidualNormArgs a, const RowPlan& p, cudaStream_t st) {
    const RowShared s = row_shared(a, p, BACKWARD, TOKEN);
    a.stages = s.stages;
    a.mod_units = s.mod_units;
    a.weight_units = s.weight_units;
    a.wsum_shared = s.wsum;
    if constexpr (BACKWARD) return launch(residual_norm_bwd_kernel<TS, TB, V, Y, WIDE, TOKEN>, a, p, s.bytes, st);
    else return launch(residual_norm_fwd_kernel<TS, TB, V, Y, WIDE, TOKEN>, a, p, s.bytes, st);
}
template <typename TS, typename TB, int V, bool WIDE, bool BACKWARD, bool TOKEN>
cudaError_t launch_y(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st) {
    return a.y.p == nullptr      ? launch_dir<TS, TB, V, 0, WIDE, BACKWARD, TOKEN>(a, p, st)
           : a.post == kNormNone ? launch_dir<TS, TB, V, 1, WIDE, BACKWARD, TOKEN>(a, p, st)
                                 : launch_dir<TS, TB, V, 2, WIDE, BACKWARD, TOKEN>(a, p, st);
}
template <typename TS, typename TB, bool BACKWARD, bool TOKEN>
cudaError_t launch_types(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st) {
    return p.team <= 32 ? launch_y<TS, TB, 1, false, BACKWARD, TOKEN>(a, p, st)
           : p.V == 1   ? launch_y<TS, TB, 1, true, BACKWARD, TOKEN>(a, p, st)
                        : launch_y<TS, TB, 2, true, BACKWARD, TOKEN>(a, p, st);
}
template <bool BACKWARD, bool TOKEN>
cudaError_t launch_rows(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st) {
    if (a.stream_dtype == kF32)
        return a.block_dtype == kF32    ? launch_types<float, float, BACKWARD, TOKEN>(a, p, st)
               : a.block_dtype == kBf16 ? launch_types<float, __nv_bfloat16, BACKWARD, TOKEN>(a, p, st)
                                        : launch_types<float, __half, BACKWARD, TOKEN>(a, p, st);
    return a.stream_dtype == kBf16 ? launch_types<__nv_bfloat16, __nv_bfloat16, BACKWARD, TOKEN>(a, p, st)
                                   : launch_types<__half, __half, BACKWARD, TOKEN>(a, p, st);
}

}  // namespace

// Each in a file of its own, which compile side by side.
cudaError_t launch_residual_norm_fwd(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_residual_norm_fwd_token(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_residual_norm_bwd(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_residual_norm_bwd_token(const ResidualNormArgs& a, const RowPlan& p, cudaStream_t st);

}  // namespace slra
