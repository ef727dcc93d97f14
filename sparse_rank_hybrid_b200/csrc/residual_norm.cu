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

constexpr int kMaxStages = 3;
constexpr size_t kRingBytes = 225 * 1024;  // dynamic shared memory of a block at most

// Threads of a block at most: the register file holds their coefficients (forward) and also their
// accumulators (backward).
constexpr int fwd_threads(int V) { return V == 1 ? 1024 : 512; }
constexpr int bwd_threads(int V) { return V == 1 ? 640 : 512; }

// Walks a worker's rows through a [B][L][C] tensor with free batch and token strides.
template <typename T>
struct RowWalk {
    T* p;
    long long step, wrap;
    __device__ RowWalk(const RowTensor& t, int b, int l, int tokens, int column)
        : p(static_cast<T*>(t.p) + b * t.b + l * t.l + column), step(t.l), wrap(t.b - tokens * t.l) {}
    __device__ void next(bool last_token) { p += step + (last_token ? wrap : 0); }
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Brings a modulation row towards the L1 before the row that needs it.
__device__ __forceinline__ void prefetch_mod(const ModTensor& m, int dtype, int b, int f, int column) {
    if (m.p) prefetch_l2(static_cast<const char*>(m.p) + (b * m.b + f * m.f + column) * (dtype == kF32 ? 4 : 2));
}

// The oldest of the ring's rows has arrived.
__device__ __forceinline__ void ring_wait(int stages) {
    if (stages == 3) async_wait<2>();
    else if (stages == 2) async_wait<1>();
    else async_wait<0>();
}

template <typename TS, typename TB, int V, bool HASY>
__global__ void __launch_bounds__(fwd_threads(V)) residual_norm_fwd_kernel(const __grid_constant__ ResidualNormArgs a) {
    constexpr int UX = kUnits<TS>, UY = HASY ? kUnits<TB> : 0, U = V * (UX + UY);
    extern __shared__ uint4 ring[];
    __shared__ float scratch[kTeamScratch];
    const int t = threadIdx.x % a.team, slots = a.channels >> 3;
    const int worker = blockIdx.x * (blockDim.x / a.team) + threadIdx.x / a.team;
    Team team{a.team, scratch, 0};
    const long long r0 = worker_lo(a.rows, a.workers, worker), r1 = worker_lo(a.rows, a.workers, worker + 1);
    const int n = static_cast<int>(r1 - r0);
    // teams of one warp take part in each other's shuffles, so they all loop as long as the longest
    const int iters = a.team <= 32 ? static_cast<int>((a.rows + a.workers - 1) / a.workers) : n;
    const int b0 = static_cast<int>(r0 / a.tokens), l0 = static_cast<int>(r0 % a.tokens), c0 = t * 8;
    const float inv = 1.0f / a.channels;

    RowWalk<const TS> px(a.x, b0, l0, a.tokens, c0);
    RowWalk<const TB> py(HASY ? a.y : a.h, b0, l0, a.tokens, c0);
    RowWalk<TS> pxo(HASY ? a.x_out : a.x, b0, l0, a.tokens, c0);
    RowWalk<TB> ph(a.norm ? a.h : a.y, b0, l0, a.tokens, c0);

    int lp = l0, left = n;  // token of the next row to copy, rows still to copy
    auto prefetch = [&](int stage) {
        if (left > 0) {
            --left;
            uint4* s = ring + static_cast<size_t>(stage) * U * blockDim.x + threadIdx.x;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (t + v * a.team >= slots) break;
                const int c = v * a.team * 8;
#pragma unroll
                for (int i = 0; i < UX; ++i)
                    async_copy16(s + (v * UX + i) * blockDim.x, reinterpret_cast<const uint4*>(px.p + c) + i);
#pragma unroll
                for (int i = 0; i < UY; ++i)
                    async_copy16(s + (V * UX + v * UY + i) * blockDim.x, reinterpret_cast<const uint4*>(py.p + c) + i);
            }
            const bool last = ++lp == a.tokens;
            if (last) lp = 0;
            px.next(last);
            py.next(last);
        }
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch(s);

    float cg[V][8], ca[V][8], cb[V][8];  // gate wp, w (1 + scale), b (1 + scale) + shift
    int b = b0, l = l0, f = l0 / a.per, group_left = 0, stage = 0;
    for (int i = 0; i < iters; ++i) {
        prefetch(stage == 0 ? a.stages - 1 : stage - 1);
        const bool row = i < n;
        if (row && group_left == 0) {  // another modulation row
            group_left = a.per - (l - f * a.per);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = c0 + v * a.team * 8;
                if (c >= a.channels) break;
                float w[8], m[8];
                if (HASY) {
                    load8_any(a.post_weight, c, a.w_dtype, 1.f, w);
                    load8_any(a.gate.p, b * a.gate.b + f * a.gate.f + c, a.mod_dtype, 1.f, m);
#pragma unroll
                    for (int e = 0; e < 8; ++e) cg[v][e] = w[e] * m[e];
                }
                if (a.norm) {
                    load8_any(a.scale.p, b * a.scale.b + f * a.scale.f + c, a.mod_dtype, 0.f, m);
                    load8_any(a.weight, c, a.w_dtype, 1.f, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) m[e] += 1.f, ca[v][e] = w[e] * m[e];
                    load8_any(a.bias, c, a.w_dtype, 0.f, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) cb[v][e] = w[e] * m[e];
                    load8_any(a.shift.p, b * a.shift.b + f * a.shift.f + c, a.mod_dtype, 0.f, m);
#pragma unroll
                    for (int e = 0; e < 8; ++e) cb[v][e] += m[e];
                }
            }
        }
        if (row && group_left == 1 && i + 1 < n) {  // the next row's modulation
            const bool wrap = l + 1 == a.tokens;
            const int nb = wrap ? b + 1 : b, nf = wrap ? 0 : f + 1;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = c0 + v * a.team * 8;
                if (c >= a.channels) break;
                if (HASY) prefetch_mod(a.gate, a.mod_dtype, nb, nf, c);
                prefetch_mod(a.scale, a.mod_dtype, nb, nf, c);
                prefetch_mod(a.shift, a.mod_dtype, nb, nf, c);
            }
        }
        ring_wait(a.stages);
        const uint4* s = ring + static_cast<size_t>(stage) * U * blockDim.x + threadIdx.x;
        if (++stage == a.stages) stage = 0;

        float o[V][8], y[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (row && t + v * a.team < slots) {
                uint4 u[UX];
#pragma unroll
                for (int k = 0; k < UX; ++k) u[k] = s[(v * UX + k) * blockDim.x];
                unpack8<TS>(u, o[v]);
                if (HASY) {
                    uint4 w[kUnits<TB>];
#pragma unroll
                    for (int k = 0; k < UY; ++k) w[k] = s[(V * UX + v * UY + k) * blockDim.x];
                    unpack8<TB>(w, y[v]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[v][e] = y[v][e] = 0.f;
            }
        }
        if (HASY) {
            float ry = 1.f;
            if (a.post) {
                float q[1] = {0.f};
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < 8; ++e) q[0] += y[v][e] * y[v][e];
                team.sum(q);
                ry = rsqrtf(q[0] * inv + a.post_eps);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!row || t + v * a.team >= slots) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[v][e] = fmaf(cg[v][e], y[v][e] * ry, a.rs * o[v][e]);
                store8(pxo.p + v * a.team * 8, o[v]);
            }
        }
        if (a.norm) {
            float m = 0.f, q[1] = {0.f};
            if (a.norm == kNormLayer) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < 8; ++e) q[0] += o[v][e];
                team.sum(q);
                m = q[0] * inv;
                q[0] = 0.f;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (t + v * a.team >= slots) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[v][e] -= m, q[0] += o[v][e] * o[v][e];
            }
            team.sum(q);
            const float r = rsqrtf(q[0] * inv + a.eps);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!row || t + v * a.team >= slots) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[v][e] = fmaf(o[v][e] * r, ca[v][e], cb[v][e]);
                store8(ph.p + v * a.team * 8, o[v]);
            }
        }
        if (row) {
            const bool last = ++l == a.tokens;
            if (last) l = 0, ++b;
            if (--group_left == 0) f = last ? 0 : f + 1;
            pxo.next(last);
            ph.next(last);
        }
    }
}

template <typename TS, typename TB, int V, bool HASY>
__global__ void __launch_bounds__(bwd_threads(V)) residual_norm_bwd_kernel(const __grid_constant__ ResidualNormArgs a) {
    constexpr int UX = kUnits<TS>, UB = kUnits<TB>;
    constexpr int U = V * (2 * UX + (HASY ? 2 : 1) * UB);  // x, dx_out, dh and y
    extern __shared__ uint4 ring[];
    __shared__ float scratch[kTeamScratch];
    const int t = threadIdx.x % a.team, slots = a.channels >> 3;
    const int worker = blockIdx.x * (blockDim.x / a.team) + threadIdx.x / a.team;
    Team team{a.team, scratch, 0};
    const long long r0 = worker_lo(a.rows, a.workers, worker), r1 = worker_lo(a.rows, a.workers, worker + 1);
    const int n = static_cast<int>(r1 - r0);
    const int iters = a.team <= 32 ? static_cast<int>((a.rows + a.workers - 1) / a.workers) : n;
    const int b0 = static_cast<int>(r0 / a.tokens), l0 = static_cast<int>(r0 % a.tokens), c0 = t * 8;
    const float inv = 1.0f / a.channels;
    const bool has_dxo = a.dx_out.p != nullptr, has_dh = a.norm != kNormNone;

    RowWalk<const TS> px(a.x, b0, l0, a.tokens, c0), pdo(a.dx_out, b0, l0, a.tokens, c0);
    RowWalk<const TB> py(a.y, b0, l0, a.tokens, c0), pdh(a.dh, b0, l0, a.tokens, c0);
    RowWalk<TS> pdx(a.dx, b0, l0, a.tokens, c0);
    RowWalk<TB> pdy(a.dy, b0, l0, a.tokens, c0);

    int lp = l0, left = n;
    auto prefetch = [&](int stage) {
        if (left > 0) {
            --left;
            uint4* s = ring + static_cast<size_t>(stage) * U * blockDim.x + threadIdx.x;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (t + v * a.team >= slots) break;
                const int c = v * a.team * 8;
#pragma unroll
                for (int i = 0; i < UX; ++i) {
                    async_copy16(s + (v * UX + i) * blockDim.x, reinterpret_cast<const uint4*>(px.p + c) + i);
                    if (has_dxo)
                        async_copy16(s + ((V + v) * UX + i) * blockDim.x, reinterpret_cast<const uint4*>(pdo.p + c) + i);
                }
#pragma unroll
                for (int i = 0; i < UB; ++i) {
                    if (has_dh)
                        async_copy16(s + (2 * V * UX + v * UB + i) * blockDim.x,
                                     reinterpret_cast<const uint4*>(pdh.p + c) + i);
                    if (HASY)
                        async_copy16(s + (2 * V * UX + (V + v) * UB + i) * blockDim.x,
                                     reinterpret_cast<const uint4*>(py.p + c) + i);
                }
            }
            const bool last = ++lp == a.tokens;
            if (last) lp = 0;
            px.next(last);
            pdo.next(last);
            py.next(last);
            pdh.next(last);
        }
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch(s);

    float cg[V][8], ca[V][8];              // gate wp, w (1 + scale)
    float p0[V][8], p1[V][8], pq[V][8];    // sums over the rows of a modulation row
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) p0[v][e] = p1[v][e] = pq[v][e] = 0.f;
    // Sums of the weights' gradients over all rows of the worker, added to at the end of each modulation
    // row: this thread's part of shared memory where it has room, else of the worker's slot in wpart.
    float* wslot = a.wpart + static_cast<long long>(worker) * 3 * a.channels + c0;
    float* wsum = wslot;
    int wk = a.channels, wv = a.team * 8, we = 1;  // strides of the sum, the vector and the element
    if (a.wsum_shared) {
        wsum = reinterpret_cast<float*>(ring + static_cast<size_t>(a.stages) * U * blockDim.x) + threadIdx.x;
        we = blockDim.x, wv = 8 * we, wk = V * wv;
    }
    if (a.wpart)
        for (int v = 0; v < V && t + v * a.team < slots; ++v)
            for (int k = 0; k < 3; ++k)
                for (int e = 0; e < 8; ++e) wsum[k * wk + v * wv + e * we] = 0.f;

    int b = b0, l = l0, f = l0 / a.per, group_left = 0, seg_rows = 0, stage = 0;
    for (int i = 0; i < iters; ++i) {
        prefetch(stage == 0 ? a.stages - 1 : stage - 1);
        const bool row = i < n;
        if (row && group_left == 0) {
            group_left = a.per - (l - f * a.per);
            seg_rows = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = c0 + v * a.team * 8;
                if (c >= a.channels) break;
                float w[8], m[8];
                if (HASY) {
                    load8_any(a.post_weight, c, a.w_dtype, 1.f, w);
                    load8_any(a.gate.p, b * a.gate.b + f * a.gate.f + c, a.mod_dtype, 1.f, m);
#pragma unroll
                    for (int e = 0; e < 8; ++e) cg[v][e] = w[e] * m[e];
                }
                load8_any(a.weight, c, a.w_dtype, 1.f, w);
                load8_any(a.scale.p, b * a.scale.b + f * a.scale.f + c, a.mod_dtype, 0.f, m);
#pragma unroll
                for (int e = 0; e < 8; ++e) ca[v][e] = w[e] * (1.f + m[e]);
            }
        }
        if (row && group_left == 1 && i + 1 < n) {
            const bool wrap = l + 1 == a.tokens;
            const int nb = wrap ? b + 1 : b, nf = wrap ? 0 : f + 1;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = c0 + v * a.team * 8;
                if (c >= a.channels) break;
                if (HASY) prefetch_mod(a.gate, a.mod_dtype, nb, nf, c);
                prefetch_mod(a.scale, a.mod_dtype, nb, nf, c);
            }
        }
        ring_wait(a.stages);
        const uint4* s = ring + static_cast<size_t>(stage) * U * blockDim.x + threadIdx.x;
        if (++stage == a.stages) stage = 0;

        float o[V][8], y[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (row && t + v * a.team < slots) {
                uint4 u[UX], w[UB];
#pragma unroll
                for (int k = 0; k < UX; ++k) u[k] = s[(v * UX + k) * blockDim.x];
                unpack8<TS>(u, o[v]);
                if (HASY) {
#pragma unroll
                    for (int k = 0; k < UB; ++k) w[k] = s[(2 * V * UX + (V + v) * UB + k) * blockDim.x];
                    unpack8<TB>(w, y[v]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) o[v][e] = y[v][e] = 0.f;
            }
        }
        float ry = 1.f;
        if (HASY && a.post) {
            float q[1] = {0.f};
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) q[0] += y[v][e] * y[v][e];
            team.sum(q);
            ry = rsqrtf(q[0] * inv + a.post_eps);
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[v][e] *= ry;
        }
        // o becomes t, the gradient reaching the sum rs x + gate wp yh
        if (has_dh) {
            float dh[V][8], q[2] = {0.f, 0.f};
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (row && t + v * a.team < slots) {
                    uint4 w[UB];
#pragma unroll
                    for (int k = 0; k < UB; ++k) w[k] = s[(2 * V * UX + v * UB + k) * blockDim.x];
                    unpack8<TB>(w, dh[v]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (HASY) o[v][e] = fmaf(cg[v][e], y[v][e], a.rs * o[v][e]);
                        q[0] += o[v][e];
                        q[1] += dh[v][e] * ca[v][e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dh[v][e] = 0.f;
                }
            }
            float m = 0.f, am = 0.f;
            if (a.norm == kNormLayer) {
                team.sum(q);
                m = q[0] * inv;
                am = q[1] * inv;
            }
            q[0] = q[1] = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!row || t + v * a.team >= slots) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    o[v][e] -= m;
                    q[0] += o[v][e] * o[v][e];
                    q[1] += o[v][e] * (dh[v][e] * ca[v][e]);
                }
            }
            team.sum(q);
            const float r = rsqrtf(q[0] * inv + a.eps);
            const float an = q[1] * r * inv;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!row || t + v * a.team >= slots) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float nrm = o[v][e] * r;
                    p0[v][e] += dh[v][e];
                    p1[v][e] = fmaf(dh[v][e], nrm, p1[v][e]);
                    o[v][e] = r * (fmaf(dh[v][e], ca[v][e], -am) - nrm * an);
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[v][e] = 0.f;
        }
        float q[1] = {0.f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!row || t + v * a.team >= slots) break;
            float d[8];
            if (has_dxo) {
                uint4 u[UX];
#pragma unroll
                for (int k = 0; k < UX; ++k) u[k] = s[((V + v) * UX + k) * blockDim.x];
                unpack8<TS>(u, d);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[v][e] += d[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = a.rs * o[v][e];
            store8(pdx.p + v * a.team * 8, d);
            if (HASY) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    pq[v][e] = fmaf(o[v][e], y[v][e], pq[v][e]);
                    o[v][e] *= cg[v][e];
                    q[0] += o[v][e] * y[v][e];
                }
            }
        }
        if (HASY) {
            float mu = 0.f;
            if (a.post) {
                team.sum(q);
                mu = q[0] * inv;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!row || t + v * a.team >= slots) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[v][e] = ry * (o[v][e] - y[v][e] * mu);
                store8(pdy.p + v * a.team * 8, o[v]);
            }
        }
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
                    const int c = c0 + v * a.team * 8;
                    if (c >= a.channels) break;
                    if (!whole && a.part) {
                        float* part = a.part + slot * 3 * a.channels + c;
                        store8(part, p0[v]);
                        store8(part + a.channels, p1[v]);
                        store8(part + 2 * a.channels, pq[v]);
                    }
                    if (whole || a.wpart) {
                        float w[8], m[8], d[8];
                        load8_any(a.weight, c, a.w_dtype, 1.f, w);
                        load8_any(a.bias, c, a.w_dtype, 0.f, m);
#pragma unroll
                        for (int e = 0; e < 8; ++e) d[e] = w[e] * p1[v][e] + m[e] * p0[v][e];
                        if (whole && a.dshift) store8(a.dshift + g + c, p0[v]);
                        if (whole && a.dscale) store8(a.dscale + g + c, d);
                        if (HASY && whole && a.dgate) {
                            load8_any(a.post_weight, c, a.w_dtype, 1.f, w);
#pragma unroll
                            for (int e = 0; e < 8; ++e) d[e] = w[e] * pq[v][e];
                            store8(a.dgate + g + c, d);
                        }
                        if (a.wpart) {
                            float* ws = wsum + v * wv;
                            load8_any(a.scale.p, b * a.scale.b + f * a.scale.f + c, a.mod_dtype, 0.f, m);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                ws[e * we] += (1.f + m[e]) * p1[v][e];
                                ws[wk + e * we] += (1.f + m[e]) * p0[v][e];
                            }
                            if (HASY) {
                                load8_any(a.gate.p, b * a.gate.b + f * a.gate.f + c, a.mod_dtype, 1.f, m);
#pragma unroll
                                for (int e = 0; e < 8; ++e) ws[2 * wk + e * we] += m[e] * pq[v][e];
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) p0[v][e] = p1[v][e] = pq[v][e] = 0.f;
                }
            }
            const bool last = ++l == a.tokens;
            if (last) l = 0, ++b;
            if (--group_left == 0) f = last ? 0 : f + 1;
            pdx.next(last);
            pdy.next(last);
        }
    }
    if (a.wpart && a.wsum_shared)
        for (int v = 0; v < V && t + v * a.team < slots; ++v)
            for (int k = 0; k < 3; ++k)
                for (int e = 0; e < 8; ++e) wslot[k * a.channels + v * a.team * 8 + e] = wsum[k * wk + v * wv + e * we];
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

// The ring gets as many stages as shared memory has room for, and the weights' sums what is left then.
template <typename TS, typename TB, int V>
cudaError_t launch_dir(ResidualNormArgs a, const RowPlan& p, bool backward, cudaStream_t st) {
    const bool y = a.y.p != nullptr;
    const int units = backward ? 2 * kUnits<TS> + (y ? 2 : 1) * kUnits<TB> : kUnits<TS> + (y ? kUnits<TB> : 0);
    const size_t stage = size_t(16) * V * units * p.threads, sums = size_t(3) * V * 32 * p.threads;
    a.stages = kMaxStages;
    while (a.stages > 1 && a.stages * stage > kRingBytes) --a.stages;
    a.wsum_shared = backward && a.wpart && a.stages * stage + sums <= kRingBytes;
    const size_t smem = a.stages * stage + (a.wsum_shared ? sums : 0);
    if (!backward)
        return y ? launch(residual_norm_fwd_kernel<TS, TB, V, true>, a, p, smem, st)
                 : launch(residual_norm_fwd_kernel<TS, TB, V, false>, a, p, smem, st);
    return y ? launch(residual_norm_bwd_kernel<TS, TB, V, true>, a, p, smem, st)
             : launch(residual_norm_bwd_kernel<TS, TB, V, false>, a, p, smem, st);
}

template <typename TS, typename TB>
cudaError_t launch_types(const ResidualNormArgs& a, const RowPlan& p, bool backward, cudaStream_t st) {
    return p.V == 1 ? launch_dir<TS, TB, 1>(a, p, backward, st) : launch_dir<TS, TB, 2>(a, p, backward, st);
}

}  // namespace

// One vector of eight channels a thread where the block holds the row, else 2; rows of up to 32 vectors
// share a block of 128 threads.  As many blocks as are resident together.
RowPlan residual_norm_plan(long long rows, int channels, bool backward) {
    RowPlan p;
    const int slots = channels / 8;
    p.V = 1;
    if (slots <= 32) {
        p.team = 1;
        while (p.team < slots) p.team *= 2;
        p.threads = 128;
    } else {
        if (slots > (backward ? bwd_threads(1) : fwd_threads(1))) p.V = 2;
        p.team = p.threads = ((slots + p.V - 1) / p.V + 31) / 32 * 32;
    }
    const int teams = p.threads / p.team;
    const int per_sm = std::max(1, (backward ? bwd_threads(1) : fwd_threads(1)) / p.threads);
    const long long want = (rows + teams - 1) / teams;
    p.blocks = static_cast<int>(std::min<long long>(want, std::min(kSMs * per_sm, kMaxWorkers / teams)));
    p.workers = p.blocks * teams;
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
