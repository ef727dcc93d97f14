// C ABI of the operators around the attention (declared in include/slra.h): argument validation and
// launches of residual_norm.cu and qk_rope.cu.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "args.cuh"

using namespace slra;

namespace {

bool known_dtype(int32_t d) { return d == SLRA_DTYPE_BF16 || d == SLRA_DTYPE_F32 || d == SLRA_DTYPE_F16; }
int64_t size_of(int32_t dtype) { return dtype == SLRA_DTYPE_F32 ? 4 : 2; }
bool positive(float x) { return x > 0.f && std::isfinite(x); }

// What a tensor covers: pieces of `run` bytes, n[i] of them at a stride of s[i] bytes in each of its dimensions
// (batch, token, head).
struct Region {
    uintptr_t at;
    int64_t run, extent, n[3], s[3];
};

Region region(const void* p, int64_t elem, const Strides& st, int64_t B, int64_t L, int64_t Hh, int64_t D) {
    return {reinterpret_cast<uintptr_t>(p), D * elem, extent_elems(st, B, L, Hh, D) * elem, {B, L, Hh},
            {st.b * elem, st.l * elem, st.h * elem}};
}
Region piece(const void* p, int64_t bytes) { return {reinterpret_cast<uintptr_t>(p), bytes, bytes, {1, 1, 1}, {0, 0, 0}}; }

// The strides of two regions, the largest first, with each one's number of steps and what it spans from there on
// inwards.
struct Meeting {
    int levels, left;  // left: places that may still be looked at
    int64_t s[6], na[6], nb[6], span_a[7], span_b[7];

    Meeting(const Region& a, const Region& b) : levels(0), left(256) {
        for (const Region* r : {&a, &b})
            for (int i = 0; i < 3; ++i) {
                if (r->n[i] == 1) continue;
                int at = 0;
                while (at < levels && s[at] > r->s[i]) ++at;
                if (at == levels || s[at] != r->s[i]) {
                    for (int j = levels++; j > at; --j) s[j] = s[j - 1], na[j] = na[j - 1], nb[j] = nb[j - 1];
                    s[at] = r->s[i];
                    na[at] = nb[at] = 1;
                }
                (r == &a ? na : nb)[at] += r->n[i] - 1;
            }
        span_a[levels] = a.run;
        span_b[levels] = b.run;
        for (int i = levels - 1; i >= 0; --i) {
            span_a[i] = span_a[i + 1] + (na[i] - 1) * s[i];
            span_b[i] = span_b[i + 1] + (nb[i] - 1) * s[i];
        }
    }
    // Whether any of the pieces meet, from level i inwards, where b's first lies d behind a's: b's step minus a's
    // takes each value k of a range, and only those that bring the spans together are followed.
    bool meet(int i, int64_t d) {
        if (d >= span_a[i] || -d >= span_b[i]) return false;
        if (i == levels) return true;
        const auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0); };
        const int64_t lo = std::max(-floor_div(span_b[i + 1] - 1 + d, s[i]), 1 - na[i]);
        const int64_t hi = std::min(floor_div(span_a[i + 1] - 1 - d, s[i]), nb[i] - 1);
        for (int64_t k = lo; k <= hi; ++k) {
            if (--left < 0) return true;  // strides that do not nest: taken as a conflict
            if (meet(i + 1, d + k * s[i])) return true;
        }
        return false;
    }
};

// Whether tokens of one stride leave room for each other, as those of a fused buffer [q | k | v] do: most views
// that meet in their extents, at a fraction of what following the strides takes.
bool tokens_interleave(const Region& a, const Region& b) {
    const int64_t s = a.s[1];
    if (a.n[1] == 1 || b.n[1] == 1 || b.s[1] != s || (a.n[0] > 1 && a.s[0] % s != 0) || (b.n[0] > 1 && b.s[0] % s != 0))
        return false;
    int64_t d = static_cast<int64_t>(b.at - a.at) % s;
    if (d < 0) d += s;
    return d >= (a.n[2] - 1) * a.s[2] + a.run && d + (b.n[2] - 1) * b.s[2] + b.run <= s;
}

bool pieces_meet(const Region& a, const Region& b) {
    return !tokens_interleave(a, b) && Meeting(a, b).meet(0, static_cast<int64_t>(b.at - a.at));
}

// Whether two regions may share a byte.  Views of one buffer whose rows, heads or samples interleave do not.
inline bool conflict(const Region& a, const Region& b) {
    if (!a.at || !b.at) return false;
    const uintptr_t ae = a.at + static_cast<uintptr_t>(a.extent), be = b.at + static_cast<uintptr_t>(b.extent);
    return a.at < be && b.at < ae && pieces_meet(a, b);
}
bool same(const Region& a, const Region& b) {
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.s[i] != b.s[i])) return false;
    return a.at == b.at && a.run == b.run;
}

// Runs body(workspace) on the caller's workspace, or on one allocated and freed on `st` where that is NULL.
template <class Body>
slra_status with_sums(size_t need, void* workspace, cudaStream_t st, Body&& body) {
    if (workspace) return body(workspace);
    void* raw = nullptr;
    if (cudaMallocAsync(&raw, need, st) != cudaSuccess) {
        cudaGetLastError();
        return SLRA_ERR_CUDA;
    }
    slra_status s = body(raw);
    if (cudaFreeAsync(raw, st) != cudaSuccess) {
        cudaGetLastError();
        if (s == SLRA_OK) s = SLRA_ERR_CUDA;
    }
    return s;
}

slra_status check_sums(size_t need, const void* workspace, size_t bytes) {
    if (!workspace) return SLRA_OK;
    return (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || bytes < need ? SLRA_ERR_WORKSPACE : SLRA_OK;
}

// ---- residual norm -------------------------------------------------------------------------------
struct Rows {
    Strides x, y, x_out, h, dx, dy;  // h stride of a row: its channels
    ModTensor gate, scale, shift;
    size_t part, wpart, bytes;  // workspace: segment sums, then the weights' sums
};

// (batch, token) strides of a [B][L][C] tensor as those of one head of C elements.
bool row_strides(const int64_t s[2], int64_t L, int64_t C, int64_t elem, Strides* out) {
    if (s[0] == 0 && s[1] == 0) {
        *out = Strides{L * C, C, C};
        return true;
    }
    const int64_t t[3] = {s[0], s[1], C};
    return strides_of(t, L, 1, C, 16 / elem, out);
}

bool mod_strides(const void* p, const int64_t s[2], int64_t groups, int64_t C, int64_t elem, ModTensor* out) {
    const int64_t b = s[0] == -1 ? groups * C : s[0], f = s[1] == -1 ? C : s[1];
    *out = ModTensor{p, b, f};
    const int64_t unit = 16 / elem, most = int64_t(1) << 36;
    return b >= 0 && f >= 0 && b % unit == 0 && f % unit == 0 && b < most && f < most;
}

slra_status derive(const slra_residual_norm* p, Rows* d) {
    if (!p || p->batch < 1 || p->tokens < 1 || p->channels < 1 || p->groups < 1) return SLRA_ERR_INVALID_ARG;
    if (p->batch >= (int64_t(1) << 31) || p->tokens >= (int64_t(1) << 31) ||
        p->batch * p->tokens >= (int64_t(1) << 31) || p->tokens % p->groups != 0)
        return SLRA_ERR_INVALID_ARG;
    if (p->norm < SLRA_NORM_NONE || p->norm > SLRA_NORM_LAYER) return SLRA_ERR_INVALID_ARG;
    if (p->post_norm != SLRA_NORM_NONE && p->post_norm != SLRA_NORM_RMS) return SLRA_ERR_INVALID_ARG;
    if (!known_dtype(p->stream_dtype) || !known_dtype(p->block_dtype) || !known_dtype(p->mod_dtype) ||
        !known_dtype(p->weight_dtype))
        return SLRA_ERR_INVALID_ARG;
    if (!positive(p->eps) || !positive(p->post_eps) || !std::isfinite(p->residual_scale)) return SLRA_ERR_INVALID_ARG;
    // vectors that nothing would use, gradients of vectors that are not there
    if (p->norm == SLRA_NORM_NONE && (p->scale || p->shift || p->weight || p->bias)) return SLRA_ERR_INVALID_ARG;
    if (p->norm != SLRA_NORM_LAYER && p->bias) return SLRA_ERR_INVALID_ARG;
    if (p->post_norm == SLRA_NORM_NONE && p->post_weight) return SLRA_ERR_INVALID_ARG;
    if ((p->dgate && !p->gate) || (p->dscale && !p->scale) || (p->dshift && !p->shift) || (p->dweight && !p->weight) ||
        (p->dbias && !p->bias) || (p->dpost_weight && !p->post_weight))
        return SLRA_ERR_INVALID_ARG;
    if (p->channels % 8 != 0 || p->channels > 8192) return SLRA_ERR_UNSUPPORTED;
    if (p->stream_dtype != SLRA_DTYPE_F32 && p->block_dtype != p->stream_dtype) return SLRA_ERR_UNSUPPORTED;
    const int64_t L = p->tokens, C = p->channels, S = size_of(p->stream_dtype), K = size_of(p->block_dtype);
    const int64_t M = size_of(p->mod_dtype);
    if (!row_strides(p->x_strides, L, C, S, &d->x) || !row_strides(p->y_strides, L, C, K, &d->y) ||
        !row_strides(p->x_out_strides, L, C, S, &d->x_out) || !row_strides(p->h_strides, L, C, K, &d->h) ||
        !row_strides(p->dx_strides, L, C, S, &d->dx) || !row_strides(p->dy_strides, L, C, K, &d->dy) ||
        !mod_strides(p->gate, p->gate_strides, p->groups, C, M, &d->gate) ||
        !mod_strides(p->scale, p->scale_strides, p->groups, C, M, &d->scale) ||
        !mod_strides(p->shift, p->shift_strides, p->groups, C, M, &d->shift))
        return SLRA_ERR_INVALID_ARG;
    for (const void* v : {p->gate, p->scale, p->shift, p->weight, p->bias, p->post_weight})
        if (!aligned16(v)) return SLRA_ERR_ALIGNMENT;
    for (const void* v : {p->dgate, p->dscale, p->dshift, p->dweight, p->dbias, p->dpost_weight})
        if (!aligned16(v)) return SLRA_ERR_ALIGNMENT;
    const RowPlan plan = residual_norm_plan(p->batch * L, static_cast<int>(C), true,
                                            p->post_norm != SLRA_NORM_NONE, p->tokens == p->groups,
                                            p->stream_dtype != SLRA_DTYPE_F32);
    const size_t one = static_cast<size_t>(plan.workers) * 3 * C * sizeof(float);
    d->part = 0;
    // nothing to join where every row has modulation vectors of its own
    d->wpart = p->tokens > p->groups && (p->dgate || p->dscale || p->dshift) ? align_up(2 * one, 256) : 0;
    d->bytes = d->wpart + (p->dweight || p->dbias || p->dpost_weight ? align_up(one, 256) : 0);
    if (d->bytes == 0) d->bytes = 256;
    return SLRA_OK;
}

Region rows_region(const slra_residual_norm* p, const void* q, int32_t dtype, const Strides& st) {
    return region(q, size_of(dtype), st, p->batch, p->tokens, 1, p->channels);
}

// The regions of the vectors of p: [0, 6) read, [6, 12) written.
void vector_regions(const slra_residual_norm* p, const Rows& d, Region out[12]) {
    const int64_t M = size_of(p->mod_dtype), W = size_of(p->weight_dtype), C = p->channels;
    const ModTensor* m[3] = {&d.gate, &d.scale, &d.shift};
    for (int i = 0; i < 3; ++i)
        out[i] = piece(m[i]->p, ((p->batch - 1) * m[i]->b + (p->groups - 1) * m[i]->f + C) * M);
    out[3] = piece(p->weight, C * W);
    out[4] = piece(p->bias, C * W);
    out[5] = piece(p->post_weight, C * W);
    const int64_t mods = p->batch * p->groups * C * 4;
    out[6] = piece(p->dgate, mods);
    out[7] = piece(p->dscale, mods);
    out[8] = piece(p->dshift, mods);
    out[9] = piece(p->dweight, C * 4);
    out[10] = piece(p->dbias, C * 4);
    out[11] = piece(p->dpost_weight, C * 4);
}

ResidualNormArgs base_args(const slra_residual_norm* p, const Rows& d, const void* x, const void* y) {
    ResidualNormArgs a;
    std::memset(&a, 0, sizeof a);
    a.x = RowTensor{const_cast<void*>(x), d.x.b, d.x.l};
    a.y = RowTensor{const_cast<void*>(y), d.y.b, d.y.l};
    a.gate = d.gate;
    a.scale = d.scale;
    a.shift = d.shift;
    a.weight = p->weight;
    a.bias = p->bias;
    a.post_weight = p->post_weight;
    a.rows = p->batch * p->tokens;
    a.tokens = static_cast<int>(p->tokens);
    a.channels = static_cast<int>(p->channels);
    a.groups = static_cast<int>(p->groups);
    a.per = static_cast<int>(p->tokens / p->groups);
    a.stream_dtype = p->stream_dtype;
    a.block_dtype = p->block_dtype;
    a.mod_dtype = p->mod_dtype;
    a.w_dtype = p->weight_dtype;
    a.norm = p->norm;
    a.post = p->post_norm;
    a.eps = p->eps;
    a.post_eps = p->post_eps;
    a.rs = p->residual_scale;
    return a;
}

// y present or not, and what then may be given.
slra_status check_residual(const slra_residual_norm* p, const void* y) {
    if (!y && (p->gate || p->post_norm != SLRA_NORM_NONE || p->residual_scale != 1.0f || p->norm == SLRA_NORM_NONE))
        return SLRA_ERR_INVALID_ARG;
    return SLRA_OK;
}

// ---- QK norm and rotation ------------------------------------------------------------------------
struct Heads {
    Strides q, k, out_q, out_k, dq, dk;
    QkRopeArgs a;  // everything but the tensors
    size_t bytes;
};

slra_status derive(const slra_qk_rope* p, Heads* d) {
    if (!p || p->batch < 1 || p->tokens < 1 || p->heads < 1 || p->kv_heads < 0 || p->head_dim < 1)
        return SLRA_ERR_INVALID_ARG;
    const int64_t most = int64_t(1) << 31;
    if (p->batch >= most || p->tokens >= most || p->batch * p->tokens >= most) return SLRA_ERR_INVALID_ARG;
    if (p->norm < SLRA_QK_NORM_NONE || p->norm > SLRA_QK_NORM_TOKEN) return SLRA_ERR_INVALID_ARG;
    if ((p->rotate != 0 && p->rotate != 1) || (p->pairing != SLRA_ROPE_INTERLEAVED && p->pairing != SLRA_ROPE_HALVES) ||
        (p->schedule != SLRA_ROPE_PER_AXIS && p->schedule != SLRA_ROPE_SHARED))
        return SLRA_ERR_INVALID_ARG;
    if (!known_dtype(p->x_dtype) || !known_dtype(p->out_dtype) || !known_dtype(p->weight_dtype) || !positive(p->eps))
        return SLRA_ERR_INVALID_ARG;
    if (!(p->theta == 0.0 || p->theta >= 1.0) || !std::isfinite(p->theta)) return SLRA_ERR_INVALID_ARG;
    if (p->norm == SLRA_QK_NORM_NONE && (!p->rotate || p->wq || p->wk)) return SLRA_ERR_INVALID_ARG;
    if ((p->dwq && !p->wq) || (p->dwk && !p->wk) || (p->wk && p->kv_heads == 0)) return SLRA_ERR_INVALID_ARG;
    if (p->rotate) {
        if (p->positions) {
            if (p->positions_stride != 0 && (p->positions_stride < 3 * p->tokens || p->positions_stride >= (int64_t(1) << 36)))
                return SLRA_ERR_INVALID_ARG;
            if ((reinterpret_cast<uintptr_t>(p->positions) & 3u) != 0) return SLRA_ERR_ALIGNMENT;
        } else {
            if (p->T < 1 || p->H < 1 || p->W < 1 || p->T >= most || p->H >= most || p->W >= most || p->first_token < 0)
                return SLRA_ERR_INVALID_ARG;
            if (p->H * p->W >= most || p->T * (p->H * p->W) >= most || p->T * (p->H * p->W) < p->tokens ||
                p->first_token > p->T * (p->H * p->W) - p->tokens)
                return SLRA_ERR_INVALID_ARG;
        }
        for (int i = 0; i < 3; ++i)
            if (p->pos_offset[i] > most || p->pos_offset[i] < -most) return SLRA_ERR_INVALID_ARG;
    }
    if (p->head_dim % 8 != 0 || p->head_dim > 256) return SLRA_ERR_UNSUPPORTED;
    int64_t g = 1;
    while (g * 8 < p->head_dim) g *= 2;
    if (p->heads > 1024 || p->kv_heads > 1024 || p->heads * g > 1024 || p->kv_heads * g > 1024) return SLRA_ERR_UNSUPPORTED;
    if (p->out_dtype != p->x_dtype && p->out_dtype != SLRA_DTYPE_F32) return SLRA_ERR_UNSUPPORTED;
    for (const void* v : {p->wq, p->wk, static_cast<const void*>(p->dwq), static_cast<const void*>(p->dwk)})
        if (!aligned16(v)) return SLRA_ERR_ALIGNMENT;

    const int64_t L = p->tokens, D = p->head_dim, hq = p->heads, hk = p->kv_heads ? p->kv_heads : 1;
    const int64_t X = 16 / size_of(p->x_dtype), O = 16 / size_of(p->out_dtype);
    if (!strides_of(p->q_strides, L, hq, D, X, &d->q) || !strides_of(p->k_strides, L, hk, D, X, &d->k) ||
        !strides_of(p->out_q_strides, L, hq, D, O, &d->out_q) || !strides_of(p->out_k_strides, L, hk, D, O, &d->out_k) ||
        !strides_of(p->dq_strides, L, hq, D, X, &d->dq) || !strides_of(p->dk_strides, L, hk, D, X, &d->dk))
        return SLRA_ERR_INVALID_ARG;
    // a token's heads within 2^31 elements
    for (const Strides* st : {&d->q, &d->out_q, &d->dq})
        if ((hq - 1) * st->h + D >= most) return SLRA_ERR_UNSUPPORTED;
    for (const Strides* st : {&d->k, &d->out_k, &d->dk})
        if ((hk - 1) * st->h + D >= most) return SLRA_ERR_UNSUPPORTED;

    QkRopeArgs& a = d->a;
    std::memset(&a, 0, sizeof a);
    a.rows = p->batch * L;
    a.tokens = static_cast<int>(L);
    a.head_dim = static_cast<int>(D);
    a.side[0].heads = static_cast<int>(p->heads);
    a.side[1].heads = static_cast<int>(p->kv_heads);
    a.side[0].weight = p->wq;
    a.side[1].weight = p->wk;
    a.H = a.W = 1;  // without a rotation no pair has an angle
    a.halves = p->pairing == SLRA_ROPE_HALVES;
    a.norm = p->norm;
    a.x_dtype = p->x_dtype;
    a.out_dtype = p->out_dtype;
    a.w_dtype = p->weight_dtype;
    a.eps = p->eps;
    if (p->rotate) {
        int64_t split[3];
        const int64_t c = D / 2, given = p->rope_split[0] + p->rope_split[1] + p->rope_split[2];
        for (int i = 0; i < 3; ++i)
            if (p->rope_split[i] < 0 || p->rope_split[i] > c) return SLRA_ERR_INVALID_ARG;
        if (given > c) return SLRA_ERR_INVALID_ARG;
        if (given == 0) {
            if (!default_split(D, p->rope_split, split)) return SLRA_ERR_INVALID_ARG;
        } else {
            for (int i = 0; i < 3; ++i) split[i] = p->rope_split[i];
        }
        // omega / 2 pi = theta^(-m / n) / 2 pi in units of 2^-64 turns: powers of one ratio an axis, in long
        // double so that their products stay below a rounding of double
        const int64_t n = split[0] + split[1] + split[2];
        const long double ln = std::log(static_cast<long double>(p->theta > 0.0 ? p->theta : 10000.0));
        const long double first = 0x1p64L / 6.283185307179586476925286767L;
        long double turns = first;
        int j = 0;
        for (int ax = 0; ax < 3; ++ax) {
            if (split[ax] == 0) continue;
            const bool shared = p->schedule == SLRA_ROPE_SHARED;
            const long double ratio = std::exp(-ln / (shared ? n : split[ax]));
            if (!shared) turns = first;
            for (int64_t m = 0; m < split[ax]; ++m, ++j, turns *= ratio) {
                a.turns[j] = static_cast<uint64_t>(turns);
                a.axis[j] = static_cast<uint8_t>(ax);
            }
        }
        const bool every = j == c && std::all_of(a.turns, a.turns + j, [](uint64_t t) { return t != 0; });
        a.rotated = every ? kRopeAll : kRopeSome;
        a.positions = p->positions;
        a.positions_b = p->positions_stride;
        a.first = p->first_token;
        a.H = static_cast<int>(p->H);
        a.W = static_cast<int>(p->W);
        for (int i = 0; i < 3; ++i) a.offset[i] = p->pos_offset[i];
    }
    d->bytes = 256;
    if (p->dwq || p->dwk) {
        const RowPlan plan = qk_rope_plan(a.rows, a.head_dim, a.side[0].heads, a.side[1].heads, a.norm, true);
        const int64_t columns =
            p->norm == SLRA_QK_NORM_TOKEN ? (p->heads + p->kv_heads) * D : (p->kv_heads ? 2 : 1) * D * plan.parts;
        d->bytes = align_up(static_cast<size_t>(plan.workers) * columns * sizeof(float), 256);
    }
    return SLRA_OK;
}

Region heads_region(const slra_qk_rope* p, const void* q, int32_t dtype, const Strides& st, int64_t heads) {
    return heads > 0 ? region(q, size_of(dtype), st, p->batch, p->tokens, heads, p->head_dim) : piece(nullptr, 0);
}
Region positions_region(const slra_qk_rope* p) {
    return piece(p->rotate ? p->positions : nullptr, ((p->batch - 1) * p->positions_stride + 3 * p->tokens) * 4);
}
Region weight_region(const slra_qk_rope* p, const void* w, int64_t heads, int64_t elem) {
    return piece(w, (p->norm == SLRA_QK_NORM_TOKEN ? heads : 1) * p->head_dim * elem);
}

}  // namespace

extern "C" {

slra_status slra_residual_norm_init(slra_residual_norm* p, int64_t batch, int64_t tokens, int64_t channels) {
    if (!p) return SLRA_ERR_INVALID_ARG;
    std::memset(p, 0, sizeof *p);
    p->batch = batch;
    p->tokens = tokens;
    p->channels = channels;
    p->groups = 1;
    p->norm = SLRA_NORM_LAYER;
    p->post_norm = SLRA_NORM_NONE;
    p->stream_dtype = p->block_dtype = SLRA_DTYPE_BF16;
    p->mod_dtype = p->weight_dtype = SLRA_DTYPE_F32;
    p->eps = p->post_eps = 1e-6f;
    p->residual_scale = 1.0f;
    for (int64_t* s : {p->gate_strides, p->scale_strides, p->shift_strides}) s[0] = s[1] = -1;
    return SLRA_OK;
}

slra_status slra_residual_norm_fwd(const slra_residual_norm* p, const void* x, const void* y, void* x_out, void* h,
                                   slra_stream_t stream) {
    Rows d;
    slra_status s = derive(p, &d);
    if (s != SLRA_OK) return s;
    if ((s = check_residual(p, y)) != SLRA_OK) return s;
    if (!x || (y != nullptr) != (x_out != nullptr) || (p->norm != SLRA_NORM_NONE) != (h != nullptr))
        return SLRA_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y) || !aligned16(x_out) || !aligned16(h)) return SLRA_ERR_ALIGNMENT;
    if (!rows_disjoint(d.x_out, p->batch, p->tokens, 1, p->channels) ||
        !rows_disjoint(d.h, p->batch, p->tokens, 1, p->channels))
        return SLRA_ERR_INVALID_ARG;
    const Region rx = rows_region(p, x, p->stream_dtype, d.x), ry = rows_region(p, y, p->block_dtype, d.y);
    const Region ro = rows_region(p, x_out, p->stream_dtype, d.x_out), rh = rows_region(p, h, p->block_dtype, d.h);
    Region vec[12];
    vector_regions(p, d, vec);
    if ((!same(ro, rx) && conflict(ro, rx)) || conflict(ro, ry) || conflict(ro, rh) || conflict(rh, rx) ||
        (!same(rh, ry) && conflict(rh, ry)))
        return SLRA_ERR_INVALID_ARG;
    for (int i = 0; i < 6; ++i)
        if (conflict(ro, vec[i]) || conflict(rh, vec[i])) return SLRA_ERR_INVALID_ARG;
    if ((s = check_device()) != SLRA_OK) return s;
    ResidualNormArgs a = base_args(p, d, x, y);
    a.x_out = RowTensor{x_out, d.x_out.b, d.x_out.l};
    a.h = RowTensor{h, d.h.b, d.h.l};
    return cuda_status(launch_residual_norm(a, false, reinterpret_cast<cudaStream_t>(stream)));
}

size_t slra_residual_norm_bwd_workspace_bytes(const slra_residual_norm* p) {
    Rows d;
    return derive(p, &d) == SLRA_OK ? d.bytes : 0;
}

slra_status slra_residual_norm_bwd(const slra_residual_norm* p, const void* x, const void* y, const void* dx_out,
                                   const void* dh, void* dx, void* dy, void* workspace, size_t workspace_bytes,
                                   slra_stream_t stream) {
    Rows d;
    slra_status s = derive(p, &d);
    if (s != SLRA_OK) return s;
    if ((s = check_residual(p, y)) != SLRA_OK) return s;
    if (!x || !dx || (y != nullptr) != (dy != nullptr) || (p->norm != SLRA_NORM_NONE) != (dh != nullptr))
        return SLRA_ERR_INVALID_ARG;
    for (const void* q : {x, y, dx_out, dh, static_cast<const void*>(dx), static_cast<const void*>(dy)})
        if (!aligned16(q)) return SLRA_ERR_ALIGNMENT;
    if (!rows_disjoint(d.dx, p->batch, p->tokens, 1, p->channels) ||
        !rows_disjoint(d.dy, p->batch, p->tokens, 1, p->channels))
        return SLRA_ERR_INVALID_ARG;
    const Region in[4] = {rows_region(p, x, p->stream_dtype, d.x), rows_region(p, y, p->block_dtype, d.y),
                          rows_region(p, dx_out, p->stream_dtype, d.x_out), rows_region(p, dh, p->block_dtype, d.h)};
    const Region rdx = rows_region(p, dx, p->stream_dtype, d.dx), rdy = rows_region(p, dy, p->block_dtype, d.dy);
    const Region ws = piece(workspace, static_cast<int64_t>(workspace_bytes));
    Region vec[12];
    vector_regions(p, d, vec);
    if (conflict(rdx, in[0]) || conflict(rdx, in[1]) || (!same(rdx, in[2]) && conflict(rdx, in[2])) ||
        conflict(rdx, in[3]) || conflict(rdy, in[0]) || conflict(rdy, in[1]) || conflict(rdy, in[2]) ||
        (!same(rdy, in[3]) && conflict(rdy, in[3])) || conflict(rdx, rdy) || conflict(rdx, ws) || conflict(rdy, ws))
        return SLRA_ERR_INVALID_ARG;
    for (int i = 0; i < 12; ++i) {
        if (conflict(rdx, vec[i]) || conflict(rdy, vec[i]) || conflict(ws, vec[i])) return SLRA_ERR_INVALID_ARG;
        if (i >= 6) {
            for (const Region& r : in)
                if (conflict(vec[i], r)) return SLRA_ERR_INVALID_ARG;
            for (int j = 0; j < i; ++j)
                if (conflict(vec[i], vec[j])) return SLRA_ERR_INVALID_ARG;
        }
    }
    for (const Region& r : in)
        if (conflict(ws, r)) return SLRA_ERR_INVALID_ARG;
    if ((s = check_sums(d.bytes, workspace, workspace_bytes)) != SLRA_OK) return s;
    if ((s = check_device()) != SLRA_OK) return s;
    ResidualNormArgs a = base_args(p, d, x, y);
    a.dx_out = RowTensor{const_cast<void*>(dx_out), d.x_out.b, d.x_out.l};
    a.dh = RowTensor{const_cast<void*>(dh), d.h.b, d.h.l};
    a.dx = RowTensor{dx, d.dx.b, d.dx.l};
    a.dy = RowTensor{dy, d.dy.b, d.dy.l};
    a.dgate = p->dgate;
    a.dscale = p->dscale;
    a.dshift = p->dshift;
    a.dweight = p->dweight;
    a.dbias = p->dbias;
    a.dpost = p->dpost_weight;
    const bool mods = p->dgate || p->dscale || p->dshift, weights = p->dweight || p->dbias || p->dpost_weight;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!mods && !weights) return cuda_status(launch_residual_norm(a, true, st));
    return with_sums(d.bytes, workspace, st, [&](void* ws_ptr) {
        uint8_t* base = static_cast<uint8_t*>(ws_ptr);
        a.part = mods ? reinterpret_cast<float*>(base + d.part) : nullptr;
        a.wpart = weights ? reinterpret_cast<float*>(base + d.wpart) : nullptr;
        return cuda_status(launch_residual_norm(a, true, st));
    });
}

slra_status slra_qk_rope_init(slra_qk_rope* p, int64_t batch, int64_t tokens, int64_t heads, int64_t head_dim) {
    if (!p) return SLRA_ERR_INVALID_ARG;
    std::memset(p, 0, sizeof *p);
    p->batch = batch;
    p->tokens = tokens;
    p->heads = heads;
    p->head_dim = head_dim;
    p->T = p->H = 1;
    p->W = tokens;
    p->theta = 10000.0;
    p->norm = SLRA_QK_NORM_NONE;
    p->rotate = 1;
    p->pairing = SLRA_ROPE_INTERLEAVED;
    p->schedule = SLRA_ROPE_PER_AXIS;
    p->x_dtype = p->out_dtype = SLRA_DTYPE_BF16;
    p->weight_dtype = SLRA_DTYPE_F32;
    p->eps = 1e-6f;
    return SLRA_OK;
}

slra_status slra_qk_rope_fwd(const slra_qk_rope* p, const void* q, const void* k, void* out_q, void* out_k,
                             slra_stream_t stream) {
    Heads d;
    slra_status s = derive(p, &d);
    if (s != SLRA_OK) return s;
    if (!q || !out_q || (k != nullptr) != (p->kv_heads > 0) || (out_k != nullptr) != (p->kv_heads > 0))
        return SLRA_ERR_INVALID_ARG;
    for (const void* t : {q, k, static_cast<const void*>(out_q), static_cast<const void*>(out_k)})
        if (!aligned16(t)) return SLRA_ERR_ALIGNMENT;
    if (!rows_disjoint(d.out_q, p->batch, p->tokens, p->heads, p->head_dim) ||
        (p->kv_heads > 0 && !rows_disjoint(d.out_k, p->batch, p->tokens, p->kv_heads, p->head_dim)))
        return SLRA_ERR_INVALID_ARG;
    const Region rq = heads_region(p, q, p->x_dtype, d.q, p->heads), rk = heads_region(p, k, p->x_dtype, d.k, p->kv_heads);
    const Region oq = heads_region(p, out_q, p->out_dtype, d.out_q, p->heads);
    const Region ok = heads_region(p, out_k, p->out_dtype, d.out_k, p->kv_heads);
    const bool q_in_place = same(oq, rq) && p->x_dtype == p->out_dtype;
    const bool k_in_place = same(ok, rk) && p->x_dtype == p->out_dtype;
    if ((!q_in_place && conflict(oq, rq)) || conflict(oq, rk) || conflict(oq, ok) || conflict(ok, rq) ||
        (!k_in_place && conflict(ok, rk)))
        return SLRA_ERR_INVALID_ARG;
    const int64_t W = size_of(p->weight_dtype);
    for (const Region& r : {positions_region(p), weight_region(p, p->wq, p->heads, W), weight_region(p, p->wk, p->kv_heads, W)})
        if (conflict(oq, r) || conflict(ok, r)) return SLRA_ERR_INVALID_ARG;
    if ((s = check_device()) != SLRA_OK) return s;
    QkRopeArgs& a = d.a;
    a.side[0].x = q;
    a.side[1].x = k;
    a.side[0].out = out_q;
    a.side[1].out = out_k;
    a.side[0].sx = d.q;
    a.side[1].sx = d.k;
    a.side[0].so = d.out_q;
    a.side[1].so = d.out_k;
    return cuda_status(launch_qk_rope(a, false, reinterpret_cast<cudaStream_t>(stream)));
}

size_t slra_qk_rope_bwd_workspace_bytes(const slra_qk_rope* p) {
    Heads d;
    return derive(p, &d) == SLRA_OK ? d.bytes : 0;
}

slra_status slra_qk_rope_bwd(const slra_qk_rope* p, const void* q, const void* k, const void* dout_q,
                             const void* dout_k, void* dq, void* dk, void* workspace, size_t workspace_bytes,
                             slra_stream_t stream) {
    Heads d;
    slra_status s = derive(p, &d);
    if (s != SLRA_OK) return s;
    const bool has_k = p->kv_heads > 0, need_x = p->norm != SLRA_QK_NORM_NONE;
    if (!dout_q || !dq || (dout_k != nullptr) != has_k || (dk != nullptr) != has_k || (k && !has_k) ||
        (need_x && (!q || (has_k && !k))))
        return SLRA_ERR_INVALID_ARG;
    for (const void* t : {q, k, dout_q, dout_k, static_cast<const void*>(dq), static_cast<const void*>(dk)})
        if (!aligned16(t)) return SLRA_ERR_ALIGNMENT;
    if (!rows_disjoint(d.dq, p->batch, p->tokens, p->heads, p->head_dim) ||
        (has_k && !rows_disjoint(d.dk, p->batch, p->tokens, p->kv_heads, p->head_dim)))
        return SLRA_ERR_INVALID_ARG;
    const Region rdq = heads_region(p, dq, p->x_dtype, d.dq, p->heads);
    const Region rdk = heads_region(p, dk, p->x_dtype, d.dk, p->kv_heads);
    const Region rgq = heads_region(p, dout_q, p->out_dtype, d.out_q, p->heads);
    const Region rgk = heads_region(p, dout_k, p->out_dtype, d.out_k, p->kv_heads);
    const bool q_in_place = same(rdq, rgq) && p->x_dtype == p->out_dtype;
    const bool k_in_place = same(rdk, rgk) && p->x_dtype == p->out_dtype;
    if ((!q_in_place && conflict(rdq, rgq)) || conflict(rdq, rgk) || conflict(rdq, rdk) || conflict(rdk, rgq) ||
        (!k_in_place && conflict(rdk, rgk)))
        return SLRA_ERR_INVALID_ARG;
    const int64_t W = size_of(p->weight_dtype);
    const Region ws = piece(workspace, static_cast<int64_t>(workspace_bytes));
    const Region dw[2] = {weight_region(p, p->dwq, p->heads, 4), weight_region(p, p->dwk, p->kv_heads, 4)};
    const Region in[5] = {need_x ? heads_region(p, q, p->x_dtype, d.q, p->heads) : piece(nullptr, 0),
                          need_x ? heads_region(p, k, p->x_dtype, d.k, p->kv_heads) : piece(nullptr, 0),
                          positions_region(p), weight_region(p, p->wq, p->heads, W),
                          weight_region(p, p->wk, p->kv_heads, W)};
    for (const Region& r : in) {
        if (conflict(rdq, r) || conflict(rdk, r) || conflict(ws, r)) return SLRA_ERR_INVALID_ARG;
        for (const Region& w : dw)
            if (conflict(w, r)) return SLRA_ERR_INVALID_ARG;
    }
    for (const Region& w : dw)
        for (const Region& r : {rdq, rdk, rgq, rgk, ws})
            if (conflict(w, r)) return SLRA_ERR_INVALID_ARG;
    if (conflict(dw[0], dw[1])) return SLRA_ERR_INVALID_ARG;
    for (const Region& r : {rdq, rdk, rgq, rgk})
        if (conflict(ws, r)) return SLRA_ERR_INVALID_ARG;
    if ((s = check_sums(d.bytes, workspace, workspace_bytes)) != SLRA_OK) return s;
    if ((s = check_device()) != SLRA_OK) return s;
    QkRopeArgs& a = d.a;
    a.side[0].x = q;
    a.side[1].x = k;
    a.side[0].d = dout_q;
    a.side[1].d = dout_k;
    a.side[0].out = dq;
    a.side[1].out = dk;
    a.side[0].sx = d.q;
    a.side[1].sx = d.k;
    a.side[0].sd = d.out_q;
    a.side[1].sd = d.out_k;
    a.side[0].so = d.dq;
    a.side[1].so = d.dk;
    a.side[0].dweight = p->dwq;
    a.side[1].dweight = p->dwk;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!p->dwq && !p->dwk) return cuda_status(launch_qk_rope(a, true, st));
    return with_sums(d.bytes, workspace, st, [&](void* ws_ptr) {
        a.part = static_cast<float*>(ws_ptr);
        return cuda_status(launch_qk_rope(a, true, st));
    });
}

}  // extern "C"
